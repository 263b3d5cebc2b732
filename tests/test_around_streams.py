"""Where the operators around the layer take memory when they run on a given stream: from that stream's
own pool, so that nothing still queued on the caller's stream can hold what they are given; what they
return is also the caller's stream's. No GPU: streams and allocations are recorded."""
import contextlib

import pytest
import torch

import block_sparse_top_fvattn_b200 as fv
from block_sparse_top_fvattn_b200 import around


class Tensor:
    """An allocation: the stream that was current, the streams that were told of its use."""

    def __init__(self, on):
        self.on, self.recorded = on, []

    def record_stream(self, stream):
        self.recorded.append(stream)

    def numel(self):
        return 1

    def element_size(self):
        return 1

    def data_ptr(self):
        return id(self)


@pytest.fixture
def world(monkeypatch):
    """current stream "caller"; what was allocated; a plan whose library call does nothing."""
    state = {"current": "caller", "made": [], "ran": []}

    @contextlib.contextmanager
    def stream(s):
        before, state["current"] = state["current"], s
        yield
        state["current"] = before

    def allocate(*args, **kw):
        t = Tensor(state["current"])
        state["made"].append(t)
        return t

    plan = object.__new__(around._Plan)
    plan.name, plan.ref, plan.device, plan.dtype, plan.nws = "call", None, None, torch.float32, 64
    plan.outs = [((1, 1, 1, 1), (1, 1, 1, 1))] * 3
    plan.run = lambda *args: state["ran"].append(args[-1])
    monkeypatch.setattr(around, "_qk_plan", lambda *a: plan)
    monkeypatch.setattr(around, "_dense_plan", lambda *a: plan)
    monkeypatch.setattr(around, "_handle", lambda device, s: s or "caller")
    state["inputs"] = [torch.zeros((1, 1, 1, 64)) for _ in range(6)]
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: state["current"])
    monkeypatch.setattr(torch, "empty", allocate)
    monkeypatch.setattr(torch, "empty_strided", allocate)
    return state


CALLS = {
    "qk_norm_rope": lambda x, **kw: fv.qk_norm_rope(x[0], x[1], **kw),
    "qk_norm_rope_bwd": lambda x, **kw: fv.qk_norm_rope_bwd(x[0], x[1], x[2], x[3], torch.ones(64), torch.ones(64), **kw),
    "dense_attn": lambda x, **kw: (fv.dense_attn(x[0], x[1], x[2], **kw),),
    "dense_attn_bwd": lambda x, **kw: fv.dense_attn_bwd(*x, **kw),
}


@pytest.mark.parametrize("name", CALLS)
def test_memory_comes_from_the_stream_that_uses_it(world, name):
    got = CALLS[name](world["inputs"], stream="side")
    assert world["made"] and world["ran"] == ["side"] and world["current"] == "caller"
    assert all(t.on == "side" for t in world["made"])
    # the caller's stream may go on using what it is given; scratch is the side stream's alone
    assert got and all("caller" in t.recorded for t in got)


@pytest.mark.parametrize("name", CALLS)
def test_memory_of_the_current_stream(world, name):
    CALLS[name](world["inputs"])
    assert world["made"] and world["ran"] == ["caller"]
    assert all(t.on == "caller" and not t.recorded for t in world["made"])
