"""The per-head norm and rotation of queries and keys, and its gradients, against the fp64 oracle.

Bounds, with f = 2^-24 and u the half step of the tensors' type: an output is a few fp32 operations
on the row's elements and its mean square (d + 8 half steps of fp32, a 2-ulp reciprocal square root):
(d + 32) f of the pair's magnitude |x r w| + |partner|, and one rounding, u |y|. Gradients: the same
of the magnitudes of their two terms; dw a sum of n terms in fp32, in runs that are joined in 64 bits."""
import ctypes

import numpy as np
import pytest
import torch

import block_sparse_top_fvattn_b200 as fv
from block_sparse_top_fvattn_b200 import _lib
from oracle import around
from dense_cases import F, HALF, f64

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fv.load()


def tables(rows, rot):
    a = np.arange(rows)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)[None, :]
    return torch.from_numpy(np.cos(a)).float().cuda(), torch.from_numpy(np.sin(a)).float().cuda()


def inputs(B, S, Hq, Hk, d, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    w = torch.randn((B, S, Hq + 2 * Hk, d), generator=g).to(dtype).cuda()
    gq = torch.randn((B, Hq, S, d), generator=g).to(dtype).cuda()
    gk = torch.randn((B, Hk, S, d), generator=g).to(dtype).cuda()
    return w[:, :, :Hq], w[:, :, Hq:Hq + Hk], gq, gk


def check(q, k, gq, gk, wq, wk, cos, sin, positions, interleaved, eps):
    opt = dict(positions=positions, interleaved=interleaved, eps=eps)
    qo, ko = fv.qk_norm_rope(q, k, wq, wk, cos, sin, **opt)
    dq, dk, dwq, dwk = fv.qk_norm_rope_bwd(gq, gk, q, k, wq, wk, cos, sin, **opt)
    B, S, _, d = q.shape
    u = HALF[q.dtype]
    pos = np.broadcast_to(np.arange(S), (B, S)) if positions is None else positions.cpu().numpy()
    cs = (None, None) if cos is None else (f64(cos), f64(sin))
    for x, w, g, y, dx, dw in ((q, wq, gq, qo, dq, dwq), (k, wk, gk, ko, dk, dwk)):
        x, g = f64(x), f64(g)
        w = np.ones(d) if w is None else f64(w)
        args = (*cs, pos, interleaved, eps)
        want = around.norm_rope(x, w, *args)
        # the magnitude of what is added: the rotation with all signs positive
        mag = around.norm_rope(np.abs(x), np.abs(w), *(None if t is None else np.abs(t) for t in cs), pos, interleaved, eps)
        mag = np.maximum(np.abs(mag), np.abs(want))
        if cs[0] is not None:
            rot = 2 * cs[0].shape[1]
            n = np.abs(around.norm_rope(x, w, None, None, pos, interleaved, eps))
            a, b = (n[..., 0:rot:2], n[..., 1:rot:2]) if interleaved else (n[..., :rot // 2], n[..., rot // 2:rot])
            full = n.copy()
            if interleaved:
                full[..., 0:rot:2] = full[..., 1:rot:2] = a + b
            else:
                full[..., :rot // 2] = full[..., rot // 2:rot] = a + b
            mag = np.maximum(mag, full)
        assert (np.abs(f64(y) - want) <= (d + 32) * F * mag + u * np.abs(want) + 1e-30).all()
        wdx, wdw = around.norm_rope_grads(g, x, w, *args)
        gt = g.transpose(0, 2, 1, 3)
        gmax = np.abs(gt).max(axis=-1, keepdims=True) * 2            # a rotated element is at most |a| + |b|
        r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        wmax = np.abs(w).max()
        term = r * gmax * wmax + np.abs(x) * r ** 3 * (gmax * wmax * np.abs(x)).mean(-1, keepdims=True)
        assert (np.abs(f64(dx) - wdx) <= 2 * (d + 32) * F * term + u * np.abs(wdx) + 1e-30).all()
        if dw is not None:
            n = x.shape[0] * x.shape[1] * x.shape[2]
            total = (gmax * np.abs(x) * r).sum(axis=(0, 1, 2))
            assert (np.abs(f64(dw) - wdw) <= (min(n, 4096) + d + 32) * F * total + 1e-30).all()
    return qo, ko, dq, dk, dwq, dwk


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", [(1, 1, 1, 1, 64), (1, 1, 1, 1, 128), (3, 1, 5, 2, 128), (2, 17, 4, 4, 64),
                                   (1, 33, 12, 3, 128), (2, 130, 3, 1, 64), (16, 1, 32, 8, 128), (1, 1000, 7, 5, 128)])
@pytest.mark.parametrize("interleaved", [True, False])
def test_sizes(shape, dtype, interleaved):
    B, S, Hq, Hk, d = shape
    x = inputs(*shape, dtype)
    wq, wk = torch.randn(d, device="cuda") + 1, torch.randn(d, device="cuda") + 1
    check(*x, wq, wk, *tables(S, d), None, interleaved, 1e-6)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("d,rot", [(64, 16), (64, 48), (128, 32), (128, 96), (128, 112), (64, 0)])
def test_partial_rotation_positions_and_weights(dtype, interleaved, d, rot):
    x = inputs(2, 45, 6, 2, d, dtype)
    cos, sin = tables(5000, rot) if rot else (None, None)
    pos = torch.randint(0, 5000, (2, 45), dtype=torch.int32, generator=torch.Generator().manual_seed(1)).cuda() \
        if rot else None
    if rot:
        pos[1, :7] = pos[0, 0]                     # the same row many times
        pos[0, 1], pos[0, 2] = 0, 4999
    for wd in (dtype, F32):
        w = [torch.randn(d, device="cuda").to(wd) for _ in range(2)]
        check(*x, *w, cos, sin, pos, interleaved, 1e-5)
    r = check(*x, None, None, cos, sin, pos, interleaved, 0.5)
    assert r[4] is None and r[5] is None


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_zero_rows_and_extremes(dtype):
    q, k, gq, gk = inputs(1, 20, 2, 2, 64, dtype)
    q[0, 3] = 0
    k[0, 5] = 0
    q[0, 7] *= 1e15
    k[0, 9] *= 1e-15
    cos, sin = tables(20, 64)
    check(q, k, gq, gk, None, None, cos, sin, None, True, 1e-6)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_into_a_cache_and_other_strides(dtype):
    B, S, Hq, Hk, d, L = 2, 3, 4, 2, 128, 40
    q, k, gq, gk = inputs(B, S, Hq, Hk, d, dtype)
    cos, sin = tables(L, d)
    pos = torch.arange(10, 10 + S, dtype=torch.int32, device="cuda").expand(B, S).contiguous()
    cache = torch.full((B, Hk, L, d), 3.0, dtype=dtype, device="cuda")
    qo = torch.full((B, S, Hq, d), 3.0, dtype=dtype, device="cuda")
    a, b = fv.qk_norm_rope(q, k, None, None, cos, sin, positions=pos, q_out=qo.transpose(1, 2),
                           k_out=cache[:, :, 10:10 + S])
    wa, wb = fv.qk_norm_rope(q, k, None, None, cos, sin, positions=pos)
    assert torch.equal(a, wa) and torch.equal(cache[:, :, 10:10 + S], wb)
    assert (cache[:, :, :10] == 3).all() and (cache[:, :, 10 + S:] == 3).all()
    # gradients into slices of one buffer
    dw = torch.full((B, S, Hq + Hk + 1, d), 3.0, dtype=dtype, device="cuda")
    fv.qk_norm_rope_bwd(gq, gk, q, k, None, None, cos, sin, positions=pos, dq=dw[:, :, :Hq], dk=dw[:, :, Hq:Hq + Hk])
    dq, dk, _, _ = fv.qk_norm_rope_bwd(gq, gk, q, k, None, None, cos, sin, positions=pos)
    assert torch.equal(dw[:, :, :Hq], dq) and torch.equal(dw[:, :, Hq:Hq + Hk], dk) and (dw[:, :, -1] == 3).all()


def test_positions_outside_the_tables():
    q, k, gq, gk = inputs(2, 5, 4, 2, 64, BF16)
    cos, sin = tables(9, 64)
    pos = torch.tensor([[0, 8, 9, 3, 4], [-1, 0, 1, 2, 2**31 - 1]], dtype=torch.int32, device="cuda")
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    qo, ko = fv.qk_norm_rope(q, k, None, None, cos, sin, positions=pos, status=status)
    bad = (pos < 0) | (pos >= 9)
    for y in (qo, ko):
        assert torch.equal(y.isnan().all(-1).all(1), bad) and torch.equal(y.isnan().any(-1).any(1), bad)
    assert status[0].item() == _lib.FVATTN_ERR_INVALID and status[1].item() == 201
    status.zero_()
    dq, dk, _, _ = fv.qk_norm_rope_bwd(gq, gk, q, k, None, None, cos, sin, positions=pos, status=status)
    for y in (dq, dk):
        assert torch.equal(y.isnan().all(-1).all(-1), bad) and torch.equal(y.isnan().any(-1).any(-1), bad)
    assert status[0].item() == _lib.FVATTN_ERR_INVALID


def test_equal_bits_captured_and_on_a_stream():
    q, k, gq, gk = inputs(2, 700, 6, 2, 128, BF16)
    cos, sin = tables(700, 64)
    w = [torch.randn(128, device="cuda") for _ in range(2)]

    def both(**kw):
        return [*fv.qk_norm_rope(q, k, *w, cos, sin, **kw), *fv.qk_norm_rope_bwd(gq, gk, q, k, *w, cos, sin, **kw)]

    want = both()
    assert all(torch.equal(a, b) for a, b in zip(want, both()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = both(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = both()
    q.neg_(), gk.mul_(2)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(both(), got))
