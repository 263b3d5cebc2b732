"""Queries, outputs and gradients of more than 2^31 elements: rows of the far end equal those of a small call."""
import pytest
import torch

import block_sparse_top_fvattn_b200 as fv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_past_32_bit_offsets(dtype):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    H, S, Sk, d = 5, (1 << 32) // (5 * 64) + 77, 40, 64            # 2^32 elements and some
    if dtype == torch.float32:
        S //= 2
    g = torch.Generator(device="cuda").manual_seed(0)
    part = torch.randn((1, H, 1000, d), generator=g, device="cuda").to(dtype)
    dpart = torch.randn((1, H, 1000, d), generator=g, device="cuda").to(dtype)
    k, v = (torch.randn((1, H, Sk, d), generator=g, device="cuda").to(dtype) for _ in range(2))
    q, dout = torch.zeros((1, H, S, d), dtype=dtype, device="cuda"), torch.zeros((1, H, S, d), dtype=dtype, device="cuda")
    q[:, :, -1000:], dout[:, :, -1000:] = part, dpart
    lse = torch.empty((1, H, S), device="cuda")
    out = fv.dense_attn(q, k, v, lse=lse)
    dq, dk, dv = fv.dense_attn_bwd(dout, q, k, v, out, lse)
    lse_small = torch.empty((1, H, 1000), device="cuda")
    small = fv.dense_attn(part, k, v, lse=lse_small)
    dq_small, dk_small, dv_small = fv.dense_attn_bwd(dpart, part, k, v, small, lse_small)
    # no cap, no mask: a row's result does not depend on its place in a tile
    assert torch.equal(out[:, :, -1000:], small) and torch.equal(lse[:, :, -1000:], lse_small)
    assert torch.equal(dq[:, :, -1000:], dq_small)
    assert (dq[:, :, :-1000] == 0).all()
    # rows with no output gradient add nothing: the sums are those of the small call in another order, terms
    # of 1000 rows each (2 x 1000 half steps of fp32) and the rounding of the result
    u = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    for a, b in ((dk, dk_small), (dv, dv_small)):
        a, b = a.double(), b.double()
        assert ((a - b).abs() <= 2 * u * b.abs() + 2000 * 2.0 ** -24 * 1000).all()
