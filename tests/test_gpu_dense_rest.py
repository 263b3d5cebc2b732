"""rest lies where out lies: the strides of dimensions of one element say nothing about that."""
import pytest
import torch

import block_sparse_top_fvattn_b200 as fv
from dense_cases import draw

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.mark.parametrize("B,H,S", [(2, 4, 1), (1, 4, 30), (2, 1, 30)])
def test_rest_and_out_with_other_strides_of_single_elements(B, H, S):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    x = draw(B, H, H, S, 100, 64, BF16)
    want = torch.empty_like(x["q"]), torch.empty_like(x["q"])
    fv.dense_attn(x["q"], x["k"], x["v"], out=want[0], rest=want[1])
    # the same places, described with other strides where a dimension has one element
    out = torch.empty_like(x["q"])
    st = [s if n > 1 else 64 * 7 for n, s in zip(out.shape, out.stride())]
    rest = torch.empty_like(x["q"])
    fv.dense_attn(x["q"], x["k"], x["v"], out=out, rest=rest.as_strided(out.shape, st))
    assert torch.equal(out, want[0]) and torch.equal(rest, want[1])
    # others still have to agree
    if S > 1 and H > 1:
        with pytest.raises(ValueError, match="rest"):
            fv.dense_attn(x["q"], x["k"], x["v"], rest=torch.empty((B, S, H, 64), dtype=BF16, device="cuda").transpose(1, 2))
