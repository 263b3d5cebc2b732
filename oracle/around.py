"""fp64 forms of the operators around the routed attention: the per-head norm with rotation and
attention over all keys with capped, biased and masked scores, each with its gradients, written
from their formulas in NumPy. The gradients are pinned to differences of the forward forms.

`dense_attention` also returns the magnitudes that rounding errors are proportional to, so that a
test can bound them element by element."""
from __future__ import annotations

import numpy as np


# ------------------------------------------------------------------ norm and rotation

def _rotate(x, cos, sin, interleaved):
    """x [..., d]; cos, sin [..., rot/2] broadcast against it."""
    rot = 2 * cos.shape[-1]
    y = x.copy()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2] = a * cos - b * sin
        y[..., 1:rot:2] = a * sin + b * cos
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2] = a * cos - b * sin
        y[..., rot // 2:rot] = a * sin + b * cos
    return y


def norm_rope(x, w, cos, sin, positions, interleaved, eps):
    """x [B, S, H, d] -> [B, H, S, d]; w [d]; cos, sin [rows, rot/2] or None; positions [B, S]."""
    r = 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    y = x * r * w
    if cos is not None:
        y = _rotate(y, cos[positions][:, :, None], sin[positions][:, :, None], interleaved)
    return y.transpose(0, 2, 1, 3)


def norm_rope_grads(dy, x, w, cos, sin, positions, interleaved, eps):
    """Gradients (dx [B, S, H, d], dw [d]) for dy [B, H, S, d]."""
    g = dy.transpose(0, 2, 1, 3)
    if cos is not None:
        g = _rotate(g, cos[positions][:, :, None], -sin[positions][:, :, None], interleaved)
    r = 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    dw = (g * x * r).sum(axis=(0, 1, 2))
    gw = g * w
    dx = r * gw - x * r ** 3 * np.mean(gw * x, axis=-1, keepdims=True)
    return dx, dw


# ------------------------------------------------------------------ attention over all keys

def visible(B, Sq, Sk, causal=False, q_start=None, prefix_len=None, kv_len=None, doc_q=None, doc_k=None):
    """Bool [B, Sq, Sk] and the positions [B, Sq]."""
    j = np.arange(Sk)[None, None, :]
    start = np.full(B, Sk - Sq) if q_start is None else np.asarray(q_start, dtype=np.int64)
    p = start[:, None] + np.arange(Sq)[None, :]
    see = np.ones((B, Sq, Sk), dtype=bool)
    if causal:
        see = j <= p[:, :, None]
        if prefix_len is not None:
            see = see | (j < np.asarray(prefix_len)[:, None, None])
    if kv_len is not None:
        see = see & (j < np.asarray(kv_len)[:, None, None])
    if doc_q is not None:
        dq, dk = np.asarray(doc_q)[:, :, None], np.asarray(doc_k)[:, None, :]
        see = see & (dq == dk) & (dq >= 0)
    return see, p


def dense_attention(q, k, v, scale=None, softcap=0.0, slopes=None, dout=None, **mask):
    """q [B, Hq, Sq, d], k, v [B, Hkv, Sk, d] (fp64). A dict with out, lse, p, cap (derivative of the
    cap) and, with dout, delta, ds, dq, dk, dv. Masked keys and queries may hold anything."""
    B, Hq, Sq, d = q.shape
    Hkv, Sk = k.shape[1], k.shape[2]
    G = Hq // Hkv
    scale = 1.0 / np.sqrt(d) if scale is None else scale
    see, p = visible(B, Sq, Sk, **mask)
    see = np.broadcast_to(see[:, None], (B, Hq, Sq, Sk))
    q = np.where(see.any(axis=(1, 3))[:, None, :, None], q, 0.0)
    used = see.any(axis=(1, 2))[:, None, :, None]
    k, v = np.where(used, k, 0.0), np.where(used, v, 0.0)
    kk, vv = np.repeat(k, G, axis=1), np.repeat(v, G, axis=1)
    s = np.einsum("bhid,bhjd->bhij", q, kk) * scale
    cap = np.ones_like(s)
    if softcap > 0:
        t = np.tanh(s / softcap)
        s, cap = softcap * t, 1.0 - t * t
    far = np.abs(p[:, None, :, None] - np.arange(Sk)[None, None, None, :])
    if slopes is not None:
        s = s - np.asarray(slopes, dtype=np.float64)[None, :, None, None] * far
    s = np.where(see, s, -np.inf)
    m = s.max(axis=-1, keepdims=True)
    m0 = np.where(np.isfinite(m), m, 0.0)
    e = np.exp(s - m0)
    total = e.sum(axis=-1, keepdims=True)
    w = e / np.where(total > 0, total, 1.0)
    with np.errstate(divide="ignore"):
        lse = (m0 + np.log(total))[..., 0]
    r = {"out": np.einsum("bhij,bhjd->bhid", w, vv), "lse": lse, "p": w, "cap": cap, "q": q, "k": kk, "v": vv,
         "far": far, "scale": scale}
    if dout is None:
        return r
    g = np.where(see.any(axis=(1, 3))[:, None, :, None], dout, 0.0)
    dp = np.einsum("bhid,bhjd->bhij", g, vv)
    delta = (w * dp).sum(axis=-1, keepdims=True)
    ds = np.where(see, w * (dp - delta) * cap * scale, 0.0)

    def shared(x):
        return x.reshape(B, Hkv, G, Sk, d).sum(axis=2)

    r.update(g=g, delta=delta[..., 0], ds=ds, dq=np.einsum("bhij,bhjd->bhid", ds, kk),
             dk=shared(np.einsum("bhij,bhid->bhjd", ds, q)), dv=shared(np.einsum("bhij,bhid->bhjd", w, g)))
    return r
