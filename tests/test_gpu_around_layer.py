"""The operators around the layer run together, as they would be used: projections through the norm and
rotation into attention over all keys and back through both gradients; prompts and then single tokens
over a cache; the layer that attends densely first and routes later. Each stage's result is held to its
own bound against the fp64 oracle on that stage's inputs as the stage before left them."""
import numpy as np
import pytest
import torch

import block_sparse_top_fvattn_b200 as fv
from block_sparse_top_fvattn_b200 import _lib
from dense_cases import F, HALF, bounds, compare, f64, reference
from oracle import around

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


def check_norm(x, w, cos, sin, pos, y):
    """y against the oracle: a few fp32 operations on a pair's elements, one rounding."""
    d = x.shape[-1]
    want = around.norm_rope(f64(x), f64(w), f64(cos), f64(sin), pos, True, 1e-6)
    n = np.abs(around.norm_rope(f64(x), f64(w), None, None, pos, True, 1e-6))
    full = np.repeat(n[..., 0::2] + n[..., 1::2], 2, axis=-1)
    assert (np.abs(f64(y) - want) <= (d + 32) * F * full + HALF[x.dtype] * np.abs(want) + 1e-30).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_projections_to_gradients(dtype):
    B, S, Hq, Hkv, d = 2, 150, 4, 2, 64
    g = torch.Generator().manual_seed(0)
    x = torch.randn((B, S, Hq + 2 * Hkv, d), generator=g).to(dtype).cuda()
    wq, wk = (1 + 0.2 * torch.randn(d, generator=g)).cuda(), (1 + 0.2 * torch.randn(d, generator=g)).cuda()
    cos, sin = tables(S, d)
    pos = np.broadcast_to(np.arange(S), (B, S))
    doc = torch.zeros((B, S), dtype=torch.int32, device="cuda")
    doc[:, 90:] = 1
    cfg = fv.AttnConfig(causal=True, softcap=15.0, doc_q=doc, doc_k=doc)
    xq, xk, xv = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:].transpose(1, 2)
    q, k = fv.qk_norm_rope(xq, xk, wq, wk, cos, sin)
    check_norm(xq, wq, cos, sin, pos, q)
    check_norm(xk, wk, cos, sin, pos, k)

    dout = torch.randn((B, Hq, S, d), generator=g).to(dtype).cuda()
    lse = torch.empty((B, Hq, S), device="cuda")
    rest = torch.empty_like(q) if dtype == BF16 else None
    got = {"out": fv.dense_attn(q, k, xv, cfg, lse=lse, rest=rest), "lse": lse}
    got["dq"], got["dk"], got["dv"] = fv.dense_attn_bwd(dout, q, k, xv, got["out"], lse, cfg, rest=rest)
    a = {"q": q, "k": k, "v": xv, "dout": dout}
    r = reference(a, cfg)
    compare(got, r, bounds(r, cfg, dtype))

    dx, _, dwq, dwk = fv.qk_norm_rope_bwd(got["dq"], got["dk"], xq, xk, wq, wk, cos, sin)
    want, want_w = around.norm_rope_grads(f64(got["dq"]), f64(xq), f64(wq), f64(cos), f64(sin), pos, True, 1e-6)
    gmax = 2 * np.abs(f64(got["dq"])).transpose(0, 2, 1, 3).max(-1, keepdims=True)
    xs = f64(xq)
    rr = 1 / np.sqrt((xs * xs).mean(-1, keepdims=True) + 1e-6)
    wmax = np.abs(f64(wq)).max()
    term = rr * gmax * wmax + np.abs(xs) * rr ** 3 * (gmax * wmax * np.abs(xs)).mean(-1, keepdims=True)
    assert (np.abs(f64(dx) - want) <= 2 * (d + 32) * F * term + HALF[dtype] * np.abs(want) + 1e-30).all()
    total = (gmax * np.abs(xs) * rr).sum(axis=(0, 1, 2))
    assert (np.abs(f64(dwq) - want_w) <= (B * S * Hq + d + 32) * F * total).all()
    assert torch.isfinite(dwk).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prompt_then_single_tokens_over_a_cache(dtype):
    # unequal prompts, padded to the longest; then tokens one at a time, each at its sequence's end
    B, Hq, Hkv, d, L = 3, 8, 2, 128, 200
    prompt = [70, 33, 129]
    g = torch.Generator().manual_seed(1)
    w = [torch.randn(d, generator=g).cuda() for _ in range(2)]
    cos, sin = tables(L, d)
    K = torch.full((B, Hkv, L, d), float("nan"), dtype=dtype, device="cuda")
    V = torch.full((B, Hkv, L, d), float("nan"), dtype=dtype, device="cuda")

    def project(S):
        x = torch.randn((B, S, Hq + 2 * Hkv, d), generator=g).to(dtype).cuda()
        return x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]

    def check(q, cfg, out):
        x = {"q": q, "k": K, "v": V, "dout": q}
        r = reference(x, cfg, grads=False)
        compare({"out": out}, r, bounds(r, cfg, dtype))

    S = max(prompt)
    xq, xk, xv = project(S)
    q, _ = fv.qk_norm_rope(xq, xk, *w, cos, sin, k_out=K[:, :, :S])
    V[:, :, :S] = xv.transpose(1, 2)
    length = torch.tensor(prompt, dtype=torch.int32, device="cuda")
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    cfg = fv.AttnConfig(causal=True, q_start=zero, kv_len=length, softcap=30.0)
    check(q, cfg, fv.dense_attn(q, K, V, cfg))
    for step in range(4):
        xq, xk, xv = project(1)
        pos = length[:, None].clone()
        q, k = fv.qk_norm_rope(xq, xk, *w, cos, sin, positions=pos)
        at = length.long()
        K[torch.arange(B), :, at] = k[:, :, 0]
        V[torch.arange(B), :, at] = xv[:, 0]
        cfg = fv.AttnConfig(causal=True, q_start=length.clone(), kv_len=length + 1, softcap=30.0)
        check(q, cfg, fv.dense_attn(q, K, V, cfg))
        length += 1


def test_layer_attends_densely_first_and_routes_later():
    B, S, H, d = 1, 1000, 2, 64
    g = torch.Generator().manual_seed(2)
    x = torch.randn((B, S, 3, H, d), generator=g).to(BF16).cuda()
    w = [torch.randn(d, generator=g).cuda() for _ in range(2)]
    cos, sin = tables(S, d)
    layer = fv.LazyRouter(fv.RouteConfig(p=0.5), refresh_every=2, dense_steps=2)
    q, k = fv.qk_norm_rope(x[:, :, 0], x[:, :, 1], *w, cos, sin)
    v = x[:, :, 2].transpose(1, 2)
    dense = fv.dense_attn(q, k, v)
    csr = fv.route(q, k, fv.RouteConfig(p=0.5))
    sparse = fv.sparse_attn(q, k, v.contiguous(), csr)
    for step in range(5):
        got = layer.from_projections(x[:, :, 0], x[:, :, 1], x[:, :, 2], step, *w, cos, sin)
        assert torch.equal(got, dense if step < 2 else sparse)
        assert layer.routed == (0 if step < 2 else 1 + (step - 2) // 2)
    assert not torch.equal(dense, sparse)
    with pytest.raises(ValueError):
        fv.LazyRouter(dense_steps=-1)


def test_dense_attention_equals_the_routed_one_that_keeps_every_block():
    # same inputs, the other path of the framework: both within the bound of the fp64 value
    B, H, S, d = 1, 2, 300, 128
    g = torch.Generator().manual_seed(3)
    x = {n: torch.randn((B, H, S, d), generator=g).to(BF16).cuda() for n in ("q", "k", "v", "dout")}
    csr = fv.route(x["q"], x["k"], fv.RouteConfig(p=1.0))
    cfg = fv.AttnConfig()
    r = reference(x, cfg, grads=False)
    b = bounds(r, cfg, BF16)
    compare({"out": fv.sparse_attn(x["q"], x["k"], x["v"], csr)}, r, b)
    compare({"out": fv.dense_attn(x["q"], x["k"], x["v"], cfg)}, r, b)


def test_binding_refuses_before_any_launch():
    def t(*s, dtype=BF16):
        return torch.zeros(s, dtype=dtype, device="cuda")

    q, k, v = t(2, 4, 10, 64), t(2, 2, 12, 64), t(2, 2, 12, 64)
    lse, out = t(2, 4, 10, dtype=F32), t(2, 4, 10, 64)
    i2 = torch.zeros(2, dtype=torch.int32, device="cuda")

    def refused(f):
        with pytest.raises((ValueError, TypeError, fv.FvattnError)):
            f()

    for bad in (t(2, 2, 12, 64, dtype=F32), t(2, 2, 11, 64), t(2, 2, 12, 64).cpu(), t(1, 2, 12, 64).expand(2, 2, 12, 64),
                t(2, 2, 12, 128)[..., ::2], t(2, 2, 64, 12).transpose(2, 3), t(2, 2, 12, 68)[..., :64]):
        refused(lambda: fv.dense_attn(q, k, bad))
        refused(lambda: fv.dense_attn(q, bad, v))
    refused(lambda: fv.dense_attn(t(2, 3, 10, 64), k, v))
    refused(lambda: fv.dense_attn(t(2, 4, 10, 96), t(2, 2, 12, 96), t(2, 2, 12, 96)))
    refused(lambda: fv.dense_attn(t(0, 4, 10, 64), t(0, 2, 12, 64), t(0, 2, 12, 64)))
    refused(lambda: fv.dense_attn(q, t(2, 2, 0, 64), t(2, 2, 0, 64)))
    refused(lambda: fv.dense_attn(q.half(), k.half(), v.half()))
    refused(lambda: fv.dense_attn(q, k, v, lse=lse[:, :, :5]))
    refused(lambda: fv.dense_attn(q, k, v, lse=lse.bfloat16()))
    refused(lambda: fv.dense_attn(q, k, v, rest=t(2, 10, 4, 64).transpose(1, 2)))
    refused(lambda: fv.dense_attn(q.float(), k.float(), v.float(), rest=out))
    refused(lambda: fv.dense_attn(q, k, v, out=t(2, 4, 10, 64, dtype=F32)))
    refused(lambda: fv.dense_attn(q, k, v, fv.AttnConfig(kv_len=i2.long())))
    refused(lambda: fv.dense_attn(q, k, v, fv.AttnConfig(kv_len=i2[:1])))
    refused(lambda: fv.dense_attn(q, k, v, fv.AttnConfig(slopes=t(2, dtype=F32))))
    refused(lambda: fv.dense_attn(q, k, v, fv.AttnConfig(doc_q=t(2, 10, dtype=torch.int32))))
    refused(lambda: fv.dense_attn(q, k, v, fv.AttnConfig(softcap=-1.0)))
    refused(lambda: fv.dense_attn(q, k, v, scale=float("nan")))
    refused(lambda: fv.dense_attn(t(1, 1, 1, 64), t(1, 1, 99999, 64), t(1, 1, 99999, 64), workspace=t(8, dtype=torch.uint8)))
    refused(lambda: fv.dense_attn_bwd(out, q, k, v, out, lse[:1]))
    refused(lambda: fv.dense_attn_bwd(out, q, k, v, out, lse, dk=t(2, 2, 11, 64)))
    refused(lambda: fv.dense_attn_bwd(t(2, 4, 1, 64).expand(2, 4, 10, 64), q, k, v, out, lse))
    # a base that is not 16-byte aligned, with a description that has been seen before
    flat = t(2 * 2 * 12 * 64 + 8)
    fv.dense_attn(q, k, flat[:-8].view(2, 2, 12, 64))
    with pytest.raises(fv.FvattnError) as e:
        fv.dense_attn(q, k, flat[4:-4].view(2, 2, 12, 64))
    assert e.value.code == _lib.FVATTN_ERR_INVALID

    x, y = t(2, 10, 4, 64), t(2, 10, 2, 64)
    cos = torch.zeros((10, 32), device="cuda")
    w = torch.ones(64, device="cuda")
    pos = torch.zeros((2, 10), dtype=torch.int32, device="cuda")
    refused(lambda: fv.qk_norm_rope(x, y[:1]))
    refused(lambda: fv.qk_norm_rope(x, y, w))
    refused(lambda: fv.qk_norm_rope(x, y, w, w.double()))
    refused(lambda: fv.qk_norm_rope(x, y, w, w, cos))
    refused(lambda: fv.qk_norm_rope(x, y, w, w, cos[:9], cos[:9]))
    refused(lambda: fv.qk_norm_rope(x, y, w, w, cos[:, :5], cos[:, :5]))
    refused(lambda: fv.qk_norm_rope(x, y, w, w, cos.bfloat16(), cos.bfloat16()))
    refused(lambda: fv.qk_norm_rope(x, y, w, w, cos, cos, positions=pos.long()))
    refused(lambda: fv.qk_norm_rope(x, y, w, w, cos, cos, positions=pos[:, :9]))
    refused(lambda: fv.qk_norm_rope(x, y, w, w, positions=pos))
    refused(lambda: fv.qk_norm_rope(x, y, eps=-1.0))
    refused(lambda: fv.qk_norm_rope(x, y, q_out=t(2, 10, 4, 64)))
    refused(lambda: fv.qk_norm_rope_bwd(x, y, x, y))
    torch.cuda.synchronize()
