"""Inputs, oracle values and error bounds shared by the GPU tests of attention over all keys.

The bounds are element by element, from the roundings that the kernels make. With f = 2^-24 (half a
step of fp32) and u = 2^-8 (bf16) or f (fp32), the half step of the inputs' type:
  score     a product of d terms in fp32: (2 d + 8) f |q|.|k| scale (twice the worst case of a sum
            in any order, for adders that truncate); the cap, the bias, the exponent's argument and
            the exponential add a few half steps of their own magnitudes, 2^-21 of the weight in all
  weight    relative error 2 max_j E_ij of the row (numerator and normaliser), and u where the
            weight is rounded to bf16 for the second product
  out       that times sum_j p |v|, a sum of Sk terms in fp32, and the rounding of out, u |out|
  delta     sum_d out dout: the error of the fp32 out before its rounding, plus what the saved out
            lost (2^-16 with rest, u without, f in fp32), times |dout|
  ds        p (dp - delta) cap' scale: the weight's relative error and u of |ds|, plus p cap' scale
            times the errors of dp (a product of d terms) and of delta
  dq dk dv  those times |k|, |q|, |dout|, sums of n terms in fp32, and the rounding of the result
"""
import numpy as np
import torch

import block_sparse_top_fvattn_b200 as fv
from oracle import around

F = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: F}


def f64(t):
    return t.detach().double().cpu().numpy()


def draw(B, Hq, Hkv, Sq, Sk, d, dtype, seed=0, spread=1.0):
    g = torch.Generator().manual_seed(seed)

    def n(*s, by=1.0):
        return (by * torch.randn(s, generator=g)).to(dtype).cuda()

    return {"q": n(B, Hq, Sq, d, by=spread), "k": n(B, Hkv, Sk, d), "v": n(B, Hkv, Sk, d),
            "dout": n(B, Hq, Sq, d)}


def reference(x, cfg, scale=None, grads=True):
    m = {n: None if getattr(cfg, n) is None else getattr(cfg, n).cpu().numpy()
         for n in ("q_start", "prefix_len", "kv_len", "doc_q", "doc_k")}
    slopes = None if cfg.slopes is None else f64(cfg.slopes)
    with np.errstate(invalid="ignore"):
        return around.dense_attention(f64(x["q"]), f64(x["k"]), f64(x["v"]), scale=scale, softcap=cfg.softcap,
                                      slopes=slopes, causal=cfg.causal, dout=f64(x["dout"]) if grads else None, **m)


def bounds(r, cfg, dtype, rest=True):
    """{output: bound} for reference r."""
    u = HALF[dtype]
    d = r["q"].shape[-1]
    Sk = r["k"].shape[2]
    qk = np.einsum("bhid,bhjd->bhij", np.abs(r["q"]), np.abs(r["k"])) * r["scale"]
    fin = np.where(np.isfinite(r["lse"]), np.abs(r["lse"]), 0.0)[..., None]
    e = (2 * d + 8) * F * qk + 8 * F * (cfg.softcap + qk + fin) + 2.0 ** -21
    if cfg.slopes is not None:
        e = e + 8 * F * np.abs(f64(cfg.slopes))[None, :, None, None] * r["far"]
    p = r["p"]
    emax = np.where(p > 0, e, 0.0).max(axis=-1, keepdims=True)
    rel = 2 * emax
    relu = rel + (u if dtype == torch.bfloat16 else 0.0)
    A = np.einsum("bhij,bhjd->bhid", p, np.abs(r["v"]))
    acc = (Sk + 8) * 2 * F
    b = {"out": (relu + acc) * A + u * np.abs(r["out"]) + 1e-30,
         "lse": (rel + acc)[..., 0] + 8 * F * fin[..., 0]}
    if "ds" in r:
        G = p.shape[1] // r["dk"].shape[1]
        g, ao = np.abs(r["g"]), np.abs(r["out"])
        kept = F if dtype == torch.float32 else (2.0 ** -16 if rest else u)
        e_delta = (((relu + acc) * A + kept * ao) * g).sum(-1) + (2 * d + 8) * F * (ao * g).sum(-1)
        e_dp = (2 * d + 8) * F * np.einsum("bhid,bhjd->bhij", g, np.abs(r["v"]))
        e_ds = np.abs(r["ds"]) * (rel + 32 * F + (u if dtype == torch.bfloat16 else 0.0)) + \
            p * r["cap"] * r["scale"] * (e_dp + e_delta[..., None])
        if cfg.softcap > 0:      # the cap's derivative 1 - t^2 is off by twice the error of t
            e_ds = e_ds + p * np.abs(r["scale"]) * (2 * e / cfg.softcap + 16 * F) * \
                np.abs(np.einsum("bhid,bhjd->bhij", r["g"], r["v"]) - r["delta"][..., None])

        def shared(x):
            B, H, S, n = x.shape
            return x.reshape(B, H // G, G, S, n).sum(axis=2)

        n_rows = p.shape[2] * G
        ads = np.abs(r["ds"])
        b["dq"] = np.einsum("bhij,bhjd->bhid", e_ds + acc * ads, np.abs(r["k"])) + u * np.abs(r["dq"]) + 1e-30
        b["dk"] = shared(np.einsum("bhij,bhid->bhjd", e_ds + (n_rows + 8) * 2 * F * ads, np.abs(r["q"]))) + \
            u * np.abs(r["dk"]) + 1e-30
        b["dv"] = shared(np.einsum("bhij,bhid->bhjd", p * (relu + (n_rows + 8) * 2 * F), g)) + u * np.abs(r["dv"]) + 1e-30
    return b


def run(x, cfg, grads=True, rest=True, **kw):
    q = x["q"]
    lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
    use_rest = grads and rest and q.dtype == torch.bfloat16
    res = torch.empty(q.shape, dtype=q.dtype, device=q.device) if use_rest else None
    got = {"out": fv.dense_attn(q, x["k"], x["v"], cfg, lse=lse, rest=res, **kw), "lse": lse}
    if grads:
        got["dq"], got["dk"], got["dv"] = fv.dense_attn_bwd(x["dout"], q, x["k"], x["v"], got["out"], lse, cfg,
                                                            rest=res, **kw)
    return got


def compare(got, r, b):
    for n, t in got.items():
        a, want = f64(t), r[n]
        assert a.shape == want.shape, n
        gone = ~np.isfinite(want)
        np.testing.assert_array_equal(a[gone], want[gone], err_msg=n)
        far = np.abs(a[~gone] - want[~gone]) / b[n][~gone]
        assert not np.isnan(far).any(), f"{n}: NaN"
        assert far.max(initial=0.0) <= 1.0, f"{n}: {far.max():.2f} times its bound"
