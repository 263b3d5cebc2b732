"""A layer on a given stream: what its steps make, dense or routed, comes from that stream's memory. No GPU:
streams and allocations are recorded."""
import contextlib

import pytest
import torch

import block_sparse_top_fvattn_b200 as fv


@pytest.mark.parametrize("dense_steps", [0, 1])
def test_everything_of_a_step_is_made_on_its_stream(monkeypatch, dense_steps):
    now, made = ["caller"], []

    class Out:
        def __init__(self):
            self.recorded = []
            made.append(now[0])

        def record_stream(self, s):
            self.recorded.append(s)

    class Side:
        device = torch.device("cpu")

    class Csr:
        B, H, S, _workspace = 1, 2, 100, None

    @contextlib.contextmanager
    def stream(s):
        before, now[0] = now[0], s
        yield
        now[0] = before

    def alloc(*a, **kw):
        made.append(now[0])
        return Csr()

    def out_of(name):
        def f(*a, out=None, stream=None, **kw):
            return out if out is not None else Out()
        return f

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: now[0])
    monkeypatch.setattr(fv, "alloc_csr", alloc)
    monkeypatch.setattr(fv, "route", lambda *a, csr, **kw: made.append(now[0]))
    monkeypatch.setattr(fv, "sparse_attn", out_of("sparse"))
    monkeypatch.setattr(fv, "dense_attn", out_of("dense"))
    q, side = torch.zeros((1, 2, 100, 64)), Side()
    layer = fv.LazyRouter(dense_steps=dense_steps)
    for step in range(3):
        o = layer(q, q, q, step, stream=side)
        assert o.recorded == ["caller"]
    given = Out()
    del made[-1]
    assert layer(q, q, q, 3, out=given, stream=side) is given and not given.recorded
    assert made and set(made) == {side} and now == ["caller"]
    del made[:]
    assert layer(q, q, q, 4).recorded == [] and set(made) == {"caller"}
    side.device = torch.device("meta")
    with pytest.raises(ValueError, match="stream"):
        layer(q, q, q, 5, stream=side)
