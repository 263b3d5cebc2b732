"""Where the routed attention may write: into a contiguous tensor of the queries' size, type and device.
Dense steps of a layer take strided outputs too; a routed one must not write over what lies between."""
import pytest
import torch

import block_sparse_top_fvattn_b200 as fv


def test_outputs_that_the_routed_attention_refuses():
    q = torch.zeros((1, 2, 6, 64), dtype=torch.bfloat16)
    for good in (torch.empty_like(q), torch.empty((2, 6, 64), dtype=q.dtype)):
        fv._check_out(good, q)
    for bad in (torch.empty((1, 6, 2, 64), dtype=q.dtype).transpose(1, 2),       # tokens first
                torch.empty((1, 2, 9, 64), dtype=q.dtype)[:, :, 3:],             # a place in a cache
                torch.empty((1, 2, 5, 64), dtype=q.dtype), torch.empty((1, 2, 6, 64)),
                torch.empty((1, 2, 6, 64), dtype=q.dtype, device="meta")):
        with pytest.raises(ValueError, match="out"):
            fv._check_out(bad, q)


@pytest.mark.gpu
def test_a_layer_refuses_a_strided_output_on_routed_steps():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn((1, 2, 500, 64), generator=g).to(torch.bfloat16).cuda() for _ in range(3))
    layer = fv.LazyRouter(fv.RouteConfig(p=0.5), dense_steps=1)
    wide = torch.full((1, 500, 3, 64), 7.0, dtype=q.dtype, device="cuda")
    out = wide[:, :, :2].transpose(1, 2)
    assert torch.equal(layer(q, k, v, 0, out=out), fv.dense_attn(q, k, v))
    before = wide.clone()
    with pytest.raises(ValueError, match="out"):
        layer(q, k, v, 1, out=out)
    torch.cuda.synchronize()
    assert torch.equal(wide, before)
    dense = torch.empty_like(q)
    assert torch.equal(layer(q, k, v, 1, out=dense), layer(q, k, v, 1))
