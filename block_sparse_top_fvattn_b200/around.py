"""The operators around the routed attention: the per-head norm and rotation that make its queries
and keys from the projections, and attention over all keys with capped, biased and masked
scores; each with its gradients. Thin bindings of fvattn_qk_norm_rope, fvattn_dense_attn and
their _bwd calls (include/fvattn.h): shapes and types are checked here and in the library, memory
comes from PyTorch, every step runs in the library's kernels on one stream.

Tensors may be strided as long as their last dimension is contiguous and the other strides are
positive multiples of 16 bytes (slices of a fused projection, places in a cache, transposed views).
"""
from __future__ import annotations

import ctypes
import dataclasses
from typing import Optional, Tuple

import torch

from . import _lib
from ._lib import FVATTN_BF16, FVATTN_F32, FvattnError, check, load

__all__ = ["qk_norm_rope", "qk_norm_rope_bwd", "AttnConfig", "dense_attn", "dense_attn_bwd"]


def _dtype(t: torch.Tensor, name: str) -> int:
    if t.dtype == torch.bfloat16:
        return FVATTN_BF16
    if t.dtype == torch.float32:
        return FVATTN_F32
    raise TypeError(f"{name}: unsupported dtype {t.dtype}; bf16 or fp32")


def _check(t: torch.Tensor, name: str, shape, like: torch.Tensor, dtype=None) -> torch.Tensor:
    """A 4-D operand: on like's device, of its dtype, the last dimension contiguous."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.device != like.device:
        raise ValueError(f"{name} is on {t.device}, not on {like.device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.dtype != (dtype or like.dtype):
        raise ValueError(f"{name} must have dtype {dtype or like.dtype}, not {t.dtype}")
    if t.dim() == 4:
        unit = 16 // t.element_size()
        if t.stride(3) != 1 or t.data_ptr() % 16 or any(
                n > 1 and (s <= 0 or s % unit) for n, s in zip(t.shape[:3], t.stride()[:3])):
            raise ValueError(f"{name}: the last dimension must be contiguous, the base and the other strides "
                             f"multiples of 16 bytes, and no dimension expanded (strides {tuple(t.stride())})")
    elif not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _strides(t: torch.Tensor, tokens_first: bool = False) -> _lib.Strides:
    """Strides of a [B, H, S, d] tensor, or of a [B, S, H, d] one (tokens_first)."""
    b, x, y, _ = t.stride()
    return _lib.Strides(b, y, x) if tokens_first else _lib.Strides(b, x, y)


class _On:
    """The device and stream of a call; scratch and outputs made in it are kept from reuse by other
    streams until the call's stream has passed them."""

    def __init__(self, like: torch.Tensor, stream: Optional[torch.cuda.Stream]):
        self.device = like.device
        self.guard = torch.cuda.device(self.device)
        if stream is not None and stream.device != self.device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {self.device}")
        self.stream = stream

    def __enter__(self):
        self.guard.__enter__()
        self.current = torch.cuda.current_stream(self.device)
        self.handle = ctypes.c_void_p((self.stream or self.current).cuda_stream)
        return self

    def __exit__(self, *exc):
        return self.guard.__exit__(*exc)

    def made(self, t: torch.Tensor) -> torch.Tensor:
        if self.stream is not None and self.stream != self.current and t.numel():
            t.record_stream(self.stream)
        return t

    def scratch(self, nbytes: int, given: Optional[torch.Tensor] = None) -> torch.Tensor:
        if given is not None:
            if not given.is_cuda or given.device != self.device or not given.is_contiguous():
                raise ValueError("workspace must be a contiguous tensor on the device of the call")
            if given.numel() * given.element_size() < nbytes:
                raise ValueError(f"workspace needs {nbytes} bytes")
            return given
        return self.made(torch.empty(nbytes, dtype=torch.uint8, device=self.device))


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _status(t: Optional[torch.Tensor], like: torch.Tensor) -> Optional[torch.Tensor]:
    return None if t is None else _check(t, "status", (4,), like, torch.int32)


# ------------------------------------------------------------------ norm and rotation

def _qk_shape(q, k, q_weight, k_weight, cos, sin, positions, interleaved, eps) -> _lib.QkShape:
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("expected q [B, S, Hq, d] and k [B, S, Hk, d]")
    B, S, Hq, d = q.shape
    dt = _dtype(q, "q")
    _check(q, "q", q.shape, q)
    _check(k, "k", (B, S, k.shape[2], d), q)
    if d not in (64, 128):
        raise FvattnError(_lib.FVATTN_ERR_UNSUPPORTED, f"head size {d}")
    if (q_weight is None) != (k_weight is None):
        raise ValueError("q_weight and k_weight: both or neither")
    wdt = FVATTN_F32
    if q_weight is not None:
        wdt = _dtype(q_weight, "q_weight")
        for t, n in ((q_weight, "q_weight"), (k_weight, "k_weight")):
            _check(t, n, (d,), q, q_weight.dtype)
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin: both or neither")
    rot = rows = 0
    if cos is not None:
        if cos.dim() != 2:
            raise ValueError("cos and sin must be [rows, rot / 2]")
        for t, n in ((cos, "cos"), (sin, "sin")):
            _check(t, n, cos.shape, q, torch.float32)
        rows, rot = cos.shape[0], 2 * cos.shape[1]
        if rot < 16 or rot > d or rot % 16:
            raise ValueError(f"rotated elements must be a multiple of 16 up to {d}, not {rot}")
        if positions is None and rows < S:
            raise ValueError(f"the tables have {rows} rows for {S} tokens")
        if rows < 1:
            raise ValueError("empty tables")
    if positions is not None:
        if cos is None:
            raise ValueError("positions without cos and sin")
        _check(positions, "positions", (B, S), q, torch.int32)
    if not 0 <= eps < float("inf"):
        raise ValueError("eps must be finite and >= 0")
    return _lib.QkShape(B, S, Hq, k.shape[2], d, dt, wdt, rot, int(bool(interleaved)), float(eps), rows)


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, q_weight: Optional[torch.Tensor] = None,
                 k_weight: Optional[torch.Tensor] = None, cos: Optional[torch.Tensor] = None,
                 sin: Optional[torch.Tensor] = None, *, positions: Optional[torch.Tensor] = None,
                 interleaved: bool = True, eps: float = 1e-6, q_out: Optional[torch.Tensor] = None,
                 k_out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """fvattn_qk_norm_rope: RMS norm of every head of the projected q [B, S, Hq, d] and
    k [B, S, Hk, d] (times q_weight, k_weight [d]; None: ones) and rotation by its token's row of
    cos, sin (fp32 [rows, rot / 2]; None: no rotation), written as [B, Hq, S, d] and [B, Hk, S, d]:
    the layout of route, sparse_attn and dense_attn.

    positions: int32 [B, S], the table row of each token (None: token s uses row s); a position
    outside the tables gives NaN rows, and FVATTN_ERR_INVALID in `status` (int32 [4], zeroed by the
    caller) when given. interleaved: pairs (2i, 2i + 1), else (i, i + rot / 2). q_out, k_out: where to
    write, e.g. a place in a cache."""
    shp = _qk_shape(q, k, q_weight, k_weight, cos, sin, positions, interleaved, eps)
    with _On(q, stream) as on:
        _status(status, q)
        if q_out is None:
            q_out = on.made(torch.empty((shp.B, shp.Hq, shp.S, shp.d), dtype=q.dtype, device=q.device))
        if k_out is None:
            k_out = on.made(torch.empty((shp.B, shp.Hk, shp.S, shp.d), dtype=q.dtype, device=q.device))
        _check(q_out, "q_out", (shp.B, shp.Hq, shp.S, shp.d), q)
        _check(k_out, "k_out", (shp.B, shp.Hk, shp.S, shp.d), q)
        shp.q, shp.k, shp.qo, shp.ko = _strides(q, True), _strides(k, True), _strides(q_out), _strides(k_out)
        check(load().fvattn_qk_norm_rope(q.data_ptr(), k.data_ptr(), ctypes.byref(shp), _ptr(q_weight),
                                         _ptr(k_weight), _ptr(cos), _ptr(sin), _ptr(positions), q_out.data_ptr(),
                                         k_out.data_ptr(), _ptr(status), on.handle), "fvattn_qk_norm_rope")
    return q_out, k_out


def qk_norm_rope_bwd(dq_out: torch.Tensor, dk_out: torch.Tensor, q: torch.Tensor, k: torch.Tensor,
                     q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                     cos: Optional[torch.Tensor] = None, sin: Optional[torch.Tensor] = None, *,
                     positions: Optional[torch.Tensor] = None, interleaved: bool = True, eps: float = 1e-6,
                     dq: Optional[torch.Tensor] = None, dk: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                     stream: Optional[torch.cuda.Stream] = None):
    """fvattn_qk_norm_rope_bwd: gradients of qk_norm_rope for the output gradients dq_out
    [B, Hq, S, d] and dk_out [B, Hk, S, d]. Returns (dq, dk, dq_weight, dk_weight): dq, dk like q, k;
    the weights' gradients in fp32, None without weights. Equal calls give equal bits."""
    shp = _qk_shape(q, k, q_weight, k_weight, cos, sin, positions, interleaved, eps)
    _check(dq_out, "dq_out", (shp.B, shp.Hq, shp.S, shp.d), q)
    _check(dk_out, "dk_out", (shp.B, shp.Hk, shp.S, shp.d), q)
    with _On(q, stream) as on:
        _status(status, q)
        if dq is None:
            dq = on.made(torch.empty(q.shape, dtype=q.dtype, device=q.device))
        if dk is None:
            dk = on.made(torch.empty(k.shape, dtype=k.dtype, device=q.device))
        _check(dq, "dq", q.shape, q)
        _check(dk, "dk", k.shape, q)
        shp.q, shp.k, shp.dq, shp.dk = _strides(q, True), _strides(k, True), _strides(dq, True), _strides(dk, True)
        shp.qo, shp.ko = _strides(dq_out), _strides(dk_out)
        dwq = dwk = None
        if q_weight is not None:
            dwq = on.made(torch.empty(shp.d, dtype=torch.float32, device=q.device))
            dwk = on.made(torch.empty(shp.d, dtype=torch.float32, device=q.device))
        lib = load()
        nws = int(lib.fvattn_qk_norm_rope_workspace_bytes(ctypes.byref(shp))) if dwq is not None else 0
        ws = on.scratch(nws, workspace)
        check(lib.fvattn_qk_norm_rope_bwd(dq_out.data_ptr(), dk_out.data_ptr(), q.data_ptr(), k.data_ptr(),
                                          ctypes.byref(shp), _ptr(q_weight), _ptr(k_weight), _ptr(cos), _ptr(sin),
                                          _ptr(positions), dq.data_ptr(), dk.data_ptr(), _ptr(dwq), _ptr(dwk),
                                          ws.data_ptr() if nws else None, nws, _ptr(status), on.handle),
              "fvattn_qk_norm_rope_bwd")
    return dq, dk, dwq, dwk


# ------------------------------------------------------------------ attention over all keys

@dataclasses.dataclass
class AttnConfig:
    """What caps, biases and masks the scores of dense_attn (fvattn_dense_shape, fvattn_dense_mask).

    softcap     c > 0: scores become c tanh(score / c); 0: none
    causal      key j is visible to the query at position p when j <= p or j < prefix_len
    slopes      fp32 [Hq]: the score falls by slope * |p - j| (after the cap)
    q_start     int32 [B]: position of each sequence's first query; None: Sk - Sq
    prefix_len  int32 [B], with causal: keys below it are visible to every query
    kv_len      int32 [B]: keys from kv_len on do not exist, whatever their memory holds
    doc_q, doc_k  int32 [B, Sq] and [B, Sk]: a query sees only keys of its document number; a negative
                number is padding, which sees nothing and is seen by nothing, whatever it holds
    """
    softcap: float = 0.0
    causal: bool = False
    slopes: Optional[torch.Tensor] = None
    q_start: Optional[torch.Tensor] = None
    prefix_len: Optional[torch.Tensor] = None
    kv_len: Optional[torch.Tensor] = None
    doc_q: Optional[torch.Tensor] = None
    doc_k: Optional[torch.Tensor] = None

    def to_c(self, q: torch.Tensor, Sk: int) -> _lib.DenseMask:
        B, Hq, Sq, _ = q.shape
        if not 0 <= self.softcap < float("inf"):
            raise ValueError("softcap must be finite and >= 0")
        if self.prefix_len is not None and not self.causal:
            raise ValueError("prefix_len needs causal=True")
        if (self.doc_q is None) != (self.doc_k is None):
            raise ValueError("doc_q and doc_k: both or neither")
        want = (("slopes", (Hq,), torch.float32), ("q_start", (B,), torch.int32), ("prefix_len", (B,), torch.int32),
                ("kv_len", (B,), torch.int32), ("doc_q", (B, Sq), torch.int32), ("doc_k", (B, Sk), torch.int32))
        for name, shape, dtype in want:
            t = getattr(self, name)
            if t is not None:
                _check(t, name, shape, q, dtype)
        return _lib.DenseMask(_ptr(self.slopes), _ptr(self.q_start), _ptr(self.kv_len), _ptr(self.prefix_len),
                              _ptr(self.doc_q), _ptr(self.doc_k))


def _dense_shape(q, k, v, cfg: AttnConfig, scale: float) -> _lib.DenseShape:
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("expected q [B, Hq, Sq, d], k and v [B, Hkv, Sk, d]")
    B, Hq, Sq, d = q.shape
    dt = _dtype(q, "q")
    _check(q, "q", q.shape, q)
    _check(k, "k", (B, k.shape[1], k.shape[2], d), q)
    _check(v, "v", k.shape, q)
    if k.shape[1] == 0 or Hq % k.shape[1]:
        raise ValueError(f"{Hq} query heads cannot share {k.shape[1]} key heads")
    shp = _lib.DenseShape(B, Hq, k.shape[1], Sq, k.shape[2], d, dt, float(scale), float(cfg.softcap),
                          int(bool(cfg.causal)))
    shp.q, shp.k, shp.v = _strides(q), _strides(k), _strides(v)
    return shp


def dense_attn(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cfg: Optional[AttnConfig] = None, *,
               out: Optional[torch.Tensor] = None, rest: Optional[torch.Tensor] = None,
               lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
               status: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None,
               scale: float = 0.0) -> torch.Tensor:
    """fvattn_dense_attn: exact attention of q [B, Hq, Sq, d] over all keys k, v [B, Hkv, Sk, d] that
    cfg leaves visible (query head h reads key head h // (Hq // Hkv)). Returns out [B, Hq, Sq, d]; a row
    that sees no key is zeros. lse: optional fp32 [B, Hq, Sq], receives log sum exp of each row's
    scores (-inf for such a row). rest: optional bf16 tensor with out's strides that receives what
    out's rounding left over; with it dense_attn_bwd is as exact as from an unrounded out. status:
    optional int32 [4] zeroed by the caller; a wait that ran out in a kernel is reported there and makes
    its rows NaN."""
    cfg = cfg or AttnConfig()
    shp = _dense_shape(q, k, v, cfg, scale)
    mask = cfg.to_c(q, k.shape[2])
    with _On(q, stream) as on:
        _status(status, q)
        if out is None:
            out = on.made(torch.empty(q.shape, dtype=q.dtype, device=q.device))
        _check(out, "out", q.shape, q)
        if rest is not None:
            _check(rest, "rest", q.shape, q)
            if q.dtype != torch.bfloat16 or rest.stride() != out.stride():
                raise ValueError("rest must be bf16 and have out's strides")
        if lse is not None:
            _check(lse, "lse", q.shape[:3], q, torch.float32)
        shp.o = _strides(out)
        lib = load()
        nws = int(lib.fvattn_dense_attn_workspace_bytes(ctypes.byref(shp), ctypes.byref(mask)))
        if nws == _lib.SIZE_ERROR:
            nws = 0                       # the call below says which argument is wrong
        ws = on.scratch(nws, workspace) if nws or workspace is not None else None
        check(lib.fvattn_dense_attn(q.data_ptr(), k.data_ptr(), v.data_ptr(), ctypes.byref(shp), ctypes.byref(mask),
                                    out.data_ptr(), _ptr(rest), _ptr(lse), _ptr(ws), nws, _ptr(status), on.handle),
              "fvattn_dense_attn")
    return out


def dense_attn_bwd(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                   lse: torch.Tensor, cfg: Optional[AttnConfig] = None, *, rest: Optional[torch.Tensor] = None,
                   dq: Optional[torch.Tensor] = None, dk: Optional[torch.Tensor] = None,
                   dv: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                   status: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None,
                   scale: float = 0.0) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """fvattn_dense_attn_bwd: gradients (dq, dk, dv) of dense_attn for the output gradient dout, from
    its inputs, out, lse and (optionally) rest, with the same cfg and scale. Shared key heads get the
    sum over their query heads. Equal calls give equal bits."""
    cfg = cfg or AttnConfig()
    shp = _dense_shape(q, k, v, cfg, scale)
    mask = cfg.to_c(q, k.shape[2])
    _check(dout, "dout", q.shape, q)
    _check(out, "out", q.shape, q)
    _check(lse, "lse", q.shape[:3], q, torch.float32)
    if rest is not None:
        _check(rest, "rest", q.shape, q)
        if q.dtype != torch.bfloat16 or rest.stride() != out.stride():
            raise ValueError("rest must be bf16 and have out's strides")
    with _On(q, stream) as on:
        _status(status, q)
        dq, dk, dv = (on.made(torch.empty(t.shape, dtype=t.dtype, device=t.device)) if g is None else g
                      for g, t in ((dq, q), (dk, k), (dv, v)))
        for g, n, t in ((dq, "dq", q), (dk, "dk", k), (dv, "dv", v)):
            _check(g, n, t.shape, q)
        shp.o, shp.dout = _strides(out), _strides(dout)
        shp.dq, shp.dk, shp.dv = _strides(dq), _strides(dk), _strides(dv)
        lib = load()
        nws = int(lib.fvattn_dense_attn_bwd_workspace_bytes(ctypes.byref(shp), ctypes.byref(mask)))
        if nws == _lib.SIZE_ERROR:
            nws = 0
        ws = on.scratch(max(nws, 16), workspace)
        check(lib.fvattn_dense_attn_bwd(dout.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                        _ptr(rest), lse.data_ptr(), ctypes.byref(shp), ctypes.byref(mask),
                                        dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), ws.data_ptr(), nws, _ptr(status),
                                        on.handle), "fvattn_dense_attn_bwd")
    return dq, dk, dv
