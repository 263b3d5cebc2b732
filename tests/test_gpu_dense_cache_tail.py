"""A cache that is longer than what the queries' positions reach, without lengths: under an order nobody
sees the keys behind the last query, so their memory may hold anything, as behind kv_len."""
import numpy as np
import pytest
import torch

import block_sparse_top_fvattn_b200 as fv
from dense_cases import bounds, compare, draw, reference, run

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fv.load()


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), 1e4])
@pytest.mark.parametrize("shape", [(3, 8, 2, 1, 500, 128), (3, 4, 4, 3, 333, 64), (3, 4, 2, 70, 300, 64),
                                   (3, 6, 2, 130, 400, 128)])
@pytest.mark.parametrize("cap", [0.0, 30.0])
def test_memory_behind_the_last_query(dtype, what, shape, cap):
    B, _, _, Sq, Sk, _ = shape
    x = draw(*shape, dtype, seed=1)
    # the last query's position inside a block, at its end, and before the first key; a prefix beyond it
    start = (101, 127 - Sq + 1, -Sq)
    prefix = (0, 0, 37)
    cfg = fv.AttnConfig(causal=True, q_start=i32(*start), prefix_len=i32(*prefix), softcap=cap)
    got = []
    for fill in (0.0, what):
        for b in range(B):
            end = max(start[b] + Sq, prefix[b])
            x["k"][b, :, end:], x["v"][b, :, end:] = fill, fill
        got.append(run(x, cfg))
    r = reference(x, cfg)
    compare(got[1], r, bounds(r, cfg, dtype))
    assert all(torch.equal(got[0][n], got[1][n]) for n in got[0])
    for b in range(B):
        end = max(start[b] + Sq, prefix[b])
        assert (got[1]["dk"][b, :, end:] == 0).all() and (got[1]["dv"][b, :, end:] == 0).all()
    assert np.isfinite(got[1]["out"].float().cpu().numpy()).all()
