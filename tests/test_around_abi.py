"""What the norm with rotation and attention over all keys refuse, on a machine without a GPU: the
library's host checks, and the binding's own."""
import ctypes

import pytest
import torch

import block_sparse_top_fvattn_b200 as fv
from block_sparse_top_fvattn_b200 import _lib

P = 4096                                   # aligned, never dereferenced on the host
INVALID, UNSUPPORTED, CAPACITY = _lib.FVATTN_ERR_INVALID, _lib.FVATTN_ERR_UNSUPPORTED, _lib.FVATTN_ERR_CAPACITY


def st(b, h, s):
    return _lib.Strides(b, h, s)


def qk(**kw):
    f = dict(B=2, S=10, Hq=4, Hk=2, d=64, dtype=0, weight_dtype=1, rot=64, interleaved=1, eps=1e-6, table_rows=10)
    names = {n: kw.pop(n) for n in ("q", "k", "qo", "ko", "dq", "dk") if n in kw}
    f.update(kw)
    s = _lib.QkShape(**f)
    for n, H in (("q", 4), ("k", 2), ("dq", 4), ("dk", 2)):
        setattr(s, n, names.get(n, st(10 * H * 64, 64, H * 64)))
    for n, H in (("qo", 4), ("ko", 2)):
        setattr(s, n, names.get(n, st(10 * H * 64, 10 * 64, 64)))
    return s


def call_qk(lib, s, q=P, k=P, wq=P, wk=P, cos=P, sin=P, pos=None, qo=P, ko=P):
    return lib.fvattn_qk_norm_rope(q, k, ctypes.byref(s), wq, wk, cos, sin, pos, qo, ko, None, None)


@pytest.mark.parametrize("bad,code", [
    (dict(B=0), INVALID), (dict(S=0), INVALID), (dict(Hq=0), INVALID), (dict(Hk=-1), INVALID), (dict(d=96), UNSUPPORTED),
    (dict(dtype=2), INVALID), (dict(weight_dtype=-1), INVALID), (dict(rot=8), UNSUPPORTED), (dict(rot=-16), INVALID),
    (dict(rot=80), INVALID), (dict(interleaved=2), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(table_rows=0), INVALID), (dict(table_rows=9), INVALID),
    (dict(q=st(2560, 64, 0)), INVALID), (dict(q=st(2560, 60, 256)), INVALID), (dict(ko=st(-1280, 640, 64)), INVALID),
    (dict(Hq=40000), UNSUPPORTED), (dict(S=(1 << 30) + 1), UNSUPPORTED),
])
def test_qk_norm_rope_rejects_on_the_host(lib, bad, code):
    assert call_qk(lib, qk(**bad)) == code


def test_qk_norm_rope_rejects_pointers(lib):
    s = qk()
    for n in ("q", "k", "qo", "ko", "cos", "sin"):
        assert call_qk(lib, s, **{n: None}) == INVALID
        assert call_qk(lib, s, **{n: P + 8}) == INVALID
    assert call_qk(lib, s, wq=P + 4) == INVALID and call_qk(lib, s, pos=P + 2) == INVALID
    nws = lib.fvattn_qk_norm_rope_workspace_bytes(ctypes.byref(s))
    assert nws > 0 and lib.fvattn_qk_norm_rope_workspace_bytes(ctypes.byref(qk(d=80))) == 0
    bwd = lambda ws, n, dq=P: lib.fvattn_qk_norm_rope_bwd(P, P, P, P, ctypes.byref(s), P, P, P, P, None, dq, P, P, P,  # noqa: E731
                                                          ws, n, None, None)
    assert bwd(P, nws - 1) == CAPACITY and bwd(None, nws) == INVALID and bwd(P, nws, None) == INVALID
    assert lib.fvattn_qk_norm_rope_workspace_bytes(ctypes.byref(qk(dq=st(1, 1, 1)))) == 0


def dense(**kw):
    names = {n: kw.pop(n) for n in ("q", "k", "v", "o", "dout", "dq", "dk", "dv") if n in kw}
    f = dict(B=2, Hq=4, Hkv=2, Sq=10, Sk=20, d=64, dtype=0, scale=0.0, softcap=0.0, causal=0)
    f.update(kw)
    s = _lib.DenseShape(**f)
    for n in ("q", "o", "dout", "dq"):
        setattr(s, n, names.get(n, st(4 * 640, 640, 64)))
    for n in ("k", "v", "dk", "dv"):
        setattr(s, n, names.get(n, st(2 * 1280, 1280, 64)))
    return s


def call_dense(lib, s, m=None, q=P, k=P, v=P, out=P, rest=None, lse=P, ws=P, n=1 << 40):
    return lib.fvattn_dense_attn(q, k, v, ctypes.byref(s), None if m is None else ctypes.byref(m), out, rest, lse, ws, n,
                                 None, None)


def call_bwd(lib, s, m=None, dout=P, q=P, k=P, v=P, out=P, rest=None, lse=P, dq=P, dk=P, dv=P, ws=P, n=1 << 40):
    return lib.fvattn_dense_attn_bwd(dout, q, k, v, out, rest, lse, ctypes.byref(s),
                                     None if m is None else ctypes.byref(m), dq, dk, dv, ws, n, None, None)


BAD = [(dict(B=0), INVALID), (dict(Hq=0), INVALID), (dict(Hkv=0), INVALID), (dict(Sq=0), INVALID), (dict(Sk=0), INVALID),
       (dict(Hq=5), INVALID), (dict(d=96), UNSUPPORTED), (dict(d=256), UNSUPPORTED), (dict(dtype=3), INVALID),
       (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(softcap=-1.0), INVALID),
       (dict(softcap=float("nan")), INVALID), (dict(softcap=float("inf")), INVALID),
       (dict(softcap=1e-30), INVALID), (dict(softcap=1e30), INVALID), (dict(causal=2), INVALID),
       (dict(Hq=130, Hkv=2), UNSUPPORTED), (dict(B=70000), UNSUPPORTED), (dict(B=40000), UNSUPPORTED), (dict(Sk=1 << 30), UNSUPPORTED),
       (dict(q=st(2560, 0, 64)), INVALID), (dict(k=st(2560, 1280, 60)), INVALID), (dict(v=st(0, 1280, 64)), INVALID),
       (dict(o=st(-2560, 640, 64)), INVALID)]


@pytest.mark.parametrize("bad,code", BAD)
def test_dense_attn_rejects_on_the_host(lib, bad, code):
    s = dense(**bad)
    assert call_dense(lib, s) == code and call_bwd(lib, s) == code
    assert lib.fvattn_dense_attn_workspace_bytes(ctypes.byref(s), None) == _lib.SIZE_ERROR
    assert lib.fvattn_dense_attn_bwd_workspace_bytes(ctypes.byref(s), None) == _lib.SIZE_ERROR


def test_dense_attn_rejects_pointers_masks_and_workspaces(lib):
    s = dense()
    for n in ("q", "k", "v", "out"):
        assert call_dense(lib, s, **{n: None}) == INVALID and call_dense(lib, s, **{n: P + 2}) == INVALID
    for n in ("dout", "q", "k", "v", "out", "lse", "dq", "dk", "dv", "ws"):
        assert call_bwd(lib, s, **{n: None}) == INVALID
    for n in ("dout", "dq", "dk", "dv"):
        assert call_bwd(lib, s, **{n: P + 2}) == INVALID
    for n in ("dout", "dq", "dk", "dv"):
        assert call_bwd(lib, dense(**{n: st(64, 0, 64)})) == INVALID
    assert call_bwd(lib, s, n=0) == CAPACITY
    assert call_dense(lib, dense(dtype=1), rest=P) == INVALID           # rest goes with bf16
    assert call_dense(lib, s, _lib.DenseMask(doc_q=P)) == INVALID       # one side's documents only
    assert call_dense(lib, s, _lib.DenseMask(prefix_len=P)) == INVALID  # a prefix without an order
    assert call_dense(lib, s, _lib.DenseMask(kv_len=P + 1)) == INVALID
    long = dense(B=1, Hq=1, Hkv=1, Sq=1, Sk=100000)
    need = lib.fvattn_dense_attn_workspace_bytes(ctypes.byref(long), None)
    assert 0 < need < 1 << 24                                           # the keys are split
    assert call_dense(lib, long, n=need - 1) == CAPACITY and call_dense(lib, long, ws=None) == INVALID
    assert call_dense(lib, long, ws=P + 16) == INVALID
    # strides of dimensions of size one are not read
    one = dense(B=1, q=st(-7, 640, 64), o=st(3, 640, 64), k=st(0, 1280, 64))
    assert lib.fvattn_dense_attn_workspace_bytes(ctypes.byref(one), None) != _lib.SIZE_ERROR


def test_binding_refuses_cpu_tensors_and_configs():
    q = torch.zeros((1, 2, 4, 64))
    with pytest.raises(ValueError):
        fv.dense_attn(q, q, q)
    with pytest.raises(ValueError):
        fv.dense_attn_bwd(q, q, q, q, q, torch.zeros((1, 2, 4)))
    with pytest.raises(ValueError):
        fv.qk_norm_rope(q, q)
    with pytest.raises(ValueError):
        fv.qk_norm_rope_bwd(q, q, q, q)
    with pytest.raises(TypeError):
        fv.dense_attn(q.half(), q.half(), q.half())
    for bad in (dict(softcap=-1.0), dict(softcap=float("nan")), dict(prefix_len=torch.zeros(1, dtype=torch.int32)),
                dict(doc_q=torch.zeros((1, 4), dtype=torch.int32))):
        with pytest.raises(ValueError):
            fv.AttnConfig(**bad).check(q, 4)
