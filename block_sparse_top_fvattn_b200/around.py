"""The operators around the routed attention: the per-head norm and rotation that make its queries
and keys from the projections, and attention over all keys with capped, biased and masked
scores; each with its gradients. Thin bindings of fvattn_qk_norm_rope, fvattn_dense_attn and
their _bwd calls (include/fvattn.h): shapes and types are checked here and in the library, memory
comes from PyTorch, every step runs in the library's kernels on one stream.

Tensors may be strided as long as their last dimension is contiguous and the other strides are
positive multiples of 16 bytes (slices of a fused projection, places in a cache, transposed views).

Every call takes `stream`: it runs there instead of on the current stream, whose work it does not wait
for. Its inputs have to be ready there, and theirs is the caller's care (record_stream) if they are freed
before it has passed; what the call makes itself is safe on both streams.

Nothing here records itself for autograd: outputs never require gradients. A training step calls the _bwd
functions itself, or from a torch.autograd.Function of its own.
"""
from __future__ import annotations

import ctypes
import dataclasses
from typing import Optional, Tuple

import torch

from . import _lib
from ._lib import FVATTN_BF16, FVATTN_F32, FVATTN_OK, FvattnError, check, load

__all__ = ["qk_norm_rope", "qk_norm_rope_bwd", "AttnConfig", "dense_attn", "dense_attn_bwd",
           "dense_attn_timeout_check", "dense_attn_bwd_timeout_check"]


def _dtype(t: torch.Tensor, name: str) -> int:
    if t.dtype == torch.bfloat16:
        return FVATTN_BF16
    if t.dtype == torch.float32:
        return FVATTN_F32
    raise TypeError(f"{name}: unsupported dtype {t.dtype}; bf16 or fp32")


def _check(t: torch.Tensor, name: str, shape, like: torch.Tensor, dtype=None) -> None:
    """An operand: on like's device, of its dtype (or the given one); a 4-D one with a contiguous last
    dimension, others contiguous. The library checks base addresses."""
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
        if t.stride(3) != 1 or any(n > 1 and (s <= 0 or s % unit) for n, s in zip(t.shape[:3], t.stride()[:3])):
            raise ValueError(f"{name}: the last dimension must be contiguous, the other strides multiples of 16 "
                             f"bytes, and no dimension expanded (strides {tuple(t.stride())})")
    elif not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _strides(t: torch.Tensor, tokens_first: bool = False) -> _lib.Strides:
    """Strides of a [B, H, S, d] tensor, or of a [B, S, H, d] one (tokens_first)."""
    b, x, y, _ = t.stride()
    return _lib.Strides(b, y, x) if tokens_first else _lib.Strides(b, x, y)


def _need(**tensors) -> None:
    for name, t in tensors.items():
        if t is None:
            raise ValueError(f"{name} must be given")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


# Checking the tensors of a call and describing them to the library takes longer than a small call
# runs, so both are done once per description (shapes, strides, types, devices and options, never
# addresses or contents) and kept here; calls over ever new lengths start it afresh now and then.
_PLANS_MOST = 512
_plans: dict = {}


def _meta(t: Optional[torch.Tensor]):
    return None if t is None else (t.shape, t.stride(), t.dtype, t.get_device())


def _keep(key, plan):
    if len(_plans) >= _PLANS_MOST:
        _plans.clear()
    _plans[key] = plan
    return plan


class _Plan:
    """A checked description of a call: the library's structures, the outputs it may have to make, scratch
    bytes."""

    def __init__(self, name, shape, device, dtype, nws=0, out_shapes=()):
        self.name, self.call, self.index = name, getattr(load(), name), device.index
        self.shape, self.ref, self.device, self.dtype, self.nws = shape, ctypes.byref(shape), device, dtype, nws
        self.outs = []
        for size in out_shapes:
            B, x, y, d = size
            self.outs.append(((B, x, y, d), (x * y * d, y * d, d, 1)))

    def make(self, i: int, stream) -> torch.Tensor:
        """Output i, dense (the quickest of torch's ways to allocate a tensor)."""
        size, stride = self.outs[i]
        return _made(torch.empty_strided, stream, size, stride, dtype=self.dtype, device=self.device)

    def run(self, *args) -> None:
        """The library's call, with the tensors' device current."""
        if torch.cuda.current_device() == self.index:
            code = self.call(*args)
        else:
            with torch.cuda.device(self.device):
                code = self.call(*args)
        if code != FVATTN_OK:
            raise FvattnError(code, self.name)


def _handle(device: torch.device, stream: Optional[torch.cuda.Stream]) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device.index)
    if stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
    return stream.cuda_stream


def _made(how, stream: Optional[torch.cuda.Stream], *args, **kw) -> torch.Tensor:
    """A tensor that a call makes. One that runs on a given stream takes it from that stream's memory: a
    block of the current stream's could still be in use by what is queued there. The current stream, the
    caller's, may use it too, so its memory is not given away before that has passed."""
    if stream is None:
        return how(*args, **kw)
    with torch.cuda.stream(stream):
        t = how(*args, **kw)
    if t.numel():
        t.record_stream(torch.cuda.current_stream(kw["device"]))
    return t


def _scratch(plan: _Plan, given: Optional[torch.Tensor], stream) -> Optional[torch.Tensor]:
    if given is not None:
        if given.device != plan.device or not given.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the device of the call")
        if given.numel() * given.element_size() < plan.nws:
            raise ValueError(f"workspace needs {plan.nws} bytes")
        return given
    if plan.nws == 0:
        return None
    return _made(torch.empty, stream, plan.nws, dtype=torch.uint8, device=plan.device)


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


def _qk_plan(q, k, q_weight, k_weight, cos, sin, positions, interleaved, eps, outs, grads, status) -> _Plan:
    """outs: q_out, k_out or their gradients; grads: dq, dk of the gradients' call, None in the other."""
    key = ("qk", _meta(q), _meta(k), _meta(q_weight), _meta(k_weight), _meta(cos), _meta(sin), _meta(positions),
           _meta(outs[0]), _meta(outs[1]), bool(interleaved), float(eps), _meta(status),
           None if grads is None else (_meta(grads[0]), _meta(grads[1])))
    plan = _plans.get(key)
    if plan is not None:
        return plan
    if grads is not None:
        _need(dq_out=outs[0], dk_out=outs[1])
    shp = _qk_shape(q, k, q_weight, k_weight, cos, sin, positions, interleaved, eps)
    if status is not None:
        _check(status, "status", (4,), q, torch.int32)
    shapes = ((shp.B, shp.Hq, shp.S, shp.d), (shp.B, shp.Hk, shp.S, shp.d))

    def strides(given, names, want, tokens_first):
        for t, name, n in zip(given, names, want):
            if t is None:                      # made by the call: dense
                yield _lib.Strides(n[1] * n[2] * n[3], *((n[3], n[2] * n[3]) if tokens_first else (n[2] * n[3], n[3])))
            else:
                _check(t, name, n, q)
                yield _strides(t, tokens_first)

    shp.q, shp.k = _strides(q, True), _strides(k, True)
    names = ("q_out", "k_out") if grads is None else ("dq_out", "dk_out")
    shp.qo, shp.ko = strides(outs, names, shapes, False)
    nws = 0
    if grads is not None:
        shp.dq, shp.dk = strides(grads, ("dq", "dk"), (q.shape, k.shape), True)
        if q_weight is not None:
            nws = int(load().fvattn_qk_norm_rope_workspace_bytes(ctypes.byref(shp)))
    name = "fvattn_qk_norm_rope" if grads is None else "fvattn_qk_norm_rope_bwd"
    return _keep(key, _Plan(name, shp, q.device, q.dtype, nws, shapes if grads is None else (q.shape, k.shape)))


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
    plan = _qk_plan(q, k, q_weight, k_weight, cos, sin, positions, interleaved, eps, (q_out, k_out), None, status)
    handle = _handle(plan.device, stream)
    if q_out is None:
        q_out = plan.make(0, stream)
    if k_out is None:
        k_out = plan.make(1, stream)
    plan.run(q.data_ptr(), k.data_ptr(), plan.ref, _ptr(q_weight), _ptr(k_weight), _ptr(cos), _ptr(sin),
             _ptr(positions), q_out.data_ptr(), k_out.data_ptr(), _ptr(status), handle)
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
    plan = _qk_plan(q, k, q_weight, k_weight, cos, sin, positions, interleaved, eps, (dq_out, dk_out), (dq, dk), status)
    handle = _handle(plan.device, stream)
    if dq is None:
        dq = plan.make(0, stream)
    if dk is None:
        dk = plan.make(1, stream)
    dwq = dwk = None
    if q_weight is not None:
        dwq = _made(torch.empty, stream, q.shape[3], dtype=torch.float32, device=plan.device)
        dwk = _made(torch.empty, stream, q.shape[3], dtype=torch.float32, device=plan.device)
    ws = _scratch(plan, workspace, stream)
    plan.run(dq_out.data_ptr(), dk_out.data_ptr(), q.data_ptr(), k.data_ptr(), plan.ref, _ptr(q_weight), _ptr(k_weight),
             _ptr(cos), _ptr(sin), _ptr(positions), dq.data_ptr(), dk.data_ptr(), _ptr(dwq), _ptr(dwk), _ptr(ws),
             plan.nws, _ptr(status), handle)
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
    kv_len      int32 [B]: keys from kv_len on do not exist, whatever their memory holds (nor, with causal, do
                those behind every query and prefix; other hidden keys have to hold numbers)
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

    def check(self, q: torch.Tensor, Sk: int) -> None:
        """Raises ValueError unless the configuration fits queries q and Sk keys."""
        B, Hq, Sq, _ = q.shape
        if self.softcap != 0 and not 1e-20 <= self.softcap <= 1e20:
            raise ValueError("softcap must be 0 or between 1e-20 and 1e20")
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

    def to_c(self) -> _lib.DenseMask:
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


def _dense_plan(q, k, v, cfg: AttnConfig, scale, out, rest, lse, status, grads) -> _Plan:
    """grads: (dout, dq, dk, dv) of the gradients' call, None in the other."""
    key = ("dense", _meta(q), _meta(k), _meta(v), _meta(out), _meta(rest), _meta(lse), _meta(status), float(scale),
           float(cfg.softcap), bool(cfg.causal), _meta(cfg.slopes), _meta(cfg.q_start), _meta(cfg.prefix_len),
           _meta(cfg.kv_len), _meta(cfg.doc_q), _meta(cfg.doc_k), None if grads is None else tuple(map(_meta, grads)))
    plan = _plans.get(key)
    if plan is not None:
        return plan
    if grads is not None:
        _need(dout=grads[0], out=out, lse=lse)
    shp = _dense_shape(q, k, v, cfg, scale)
    cfg.check(q, k.shape[2])
    if status is not None:
        _check(status, "status", (4,), q, torch.int32)
    if lse is not None:
        _check(lse, "lse", q.shape[:3], q, torch.float32)

    def strides(t, name, like):
        if t is None:                          # made by the call: dense
            _, H, S, d = like.shape
            return _lib.Strides(H * S * d, S * d, d)
        _check(t, name, like.shape, q)
        return _strides(t)

    shp.o = strides(out, "out", q)
    if rest is not None:
        r = strides(rest, "rest", q)
        o = shp.o
        if q.dtype != torch.bfloat16 or any(n > 1 and x != y for n, x, y in
                                            zip(q.shape, (r.b, r.h, r.s), (o.b, o.h, o.s))):
            raise ValueError("rest must be bf16 and have out's strides")
    lib = load()
    name = "fvattn_dense_attn" if grads is None else "fvattn_dense_attn_bwd"
    mask = ctypes.byref(cfg.to_c())
    if grads is None:
        nws = int(lib.fvattn_dense_attn_workspace_bytes(ctypes.byref(shp), mask))
    else:
        for n, t, like in zip(("dout", "dq", "dk", "dv"), grads, (q, q, k, v)):
            setattr(shp, n, strides(t, n, like))
        nws = int(lib.fvattn_dense_attn_bwd_workspace_bytes(ctypes.byref(shp), mask))
    if nws == _lib.SIZE_ERROR:
        # the call that follows says what is wrong
        return _Plan(name, shp, q.device, q.dtype, 0, (q.shape, k.shape, v.shape))
    return _keep(key, _Plan(name, shp, q.device, q.dtype, nws, (q.shape, k.shape, v.shape)))


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
    plan = _dense_plan(q, k, v, cfg, scale, out, rest, lse, status, None)
    handle = _handle(plan.device, stream)
    if out is None:
        out = plan.make(0, stream)
    ws = _scratch(plan, workspace, stream)
    plan.run(q.data_ptr(), k.data_ptr(), v.data_ptr(), plan.ref, ctypes.byref(cfg.to_c()), out.data_ptr(), _ptr(rest),
             _ptr(lse), _ptr(ws), plan.nws, _ptr(status), handle)
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
    plan = _dense_plan(q, k, v, cfg, scale, out, rest, lse, status, (dout, dq, dk, dv))
    handle = _handle(plan.device, stream)
    dq = plan.make(0, stream) if dq is None else dq
    dk = plan.make(1, stream) if dk is None else dk
    dv = plan.make(2, stream) if dv is None else dv
    ws = _scratch(plan, workspace, stream)
    plan.run(dout.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), _ptr(rest), lse.data_ptr(),
             plan.ref, ctypes.byref(cfg.to_c()), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), _ptr(ws), plan.nws,
             _ptr(status), handle)
    return dq, dk, dv


def dense_attn_timeout_check(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cfg: Optional[AttnConfig] = None, *,
                             step: int = 0, polls: int = 64, scale: float = 0.0):
    """fvattn_dense_attn_timeout_check: dense_attn (bf16) whose waits run out on purpose at each CTA's step
    `step`. Returns (the device status word afterwards, its detail, out, lse): FVATTN_ERR_TIMEOUT and NaN
    rows where a CTA had that many steps."""
    cfg = cfg or AttnConfig()
    lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
    status = torch.zeros(4, dtype=torch.int32, device=q.device)
    plan = _dense_plan(q, k, v, cfg, scale, None, None, lse, status, None)
    out, ws = plan.make(0, None), _scratch(plan, None, None)
    with torch.cuda.device(plan.device):
        check(load().fvattn_dense_attn_timeout_check(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), plan.ref, ctypes.byref(cfg.to_c()), out.data_ptr(), None,
            lse.data_ptr(), _ptr(ws), plan.nws, status.data_ptr(), int(step), int(polls), _handle(plan.device, None)),
            "fvattn_dense_attn_timeout_check")
    code, detail = status[:2].tolist()
    return code, detail, out, lse


def dense_attn_bwd_timeout_check(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                                 lse: torch.Tensor, cfg: Optional[AttnConfig] = None, *, step: int = 0, polls: int = 64,
                                 scale: float = 0.0):
    """fvattn_dense_attn_bwd_timeout_check: the same of dense_attn_bwd. Returns (status word, detail, dq, dk,
    dv)."""
    cfg = cfg or AttnConfig()
    status = torch.zeros(4, dtype=torch.int32, device=q.device)
    plan = _dense_plan(q, k, v, cfg, scale, out, None, lse, status, (dout, None, None, None))
    dq, dk, dv = (plan.make(i, None) for i in range(3))
    ws = _scratch(plan, None, None)
    with torch.cuda.device(plan.device):
        check(load().fvattn_dense_attn_bwd_timeout_check(
            dout.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), None, lse.data_ptr(), plan.ref,
            ctypes.byref(cfg.to_c()), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), _ptr(ws), plan.nws, status.data_ptr(),
            int(step), int(polls), _handle(plan.device, None)), "fvattn_dense_attn_bwd_timeout_check")
    code, detail = status[:2].tolist()
    return code, detail, dq, dk, dv
