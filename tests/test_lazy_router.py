"""When LazyRouter routes: its schedule over several generations, with the launches replaced by
records of what they were called on (no GPU needed)."""
import pytest
import torch

import block_sparse_top_fvattn_b200 as fv


class Csr:
    def __init__(self, B, H, S):
        self.B, self.H, self.S, self._workspace = B, H, S, object()


@pytest.fixture
def calls(monkeypatch):
    """What a layer does at each step: ("dense",), or ("sparse", number of the routing it uses)."""
    log, routings = [], []

    def route(q, k, cfg, *, csr, workspace=None, stream=None):
        routings.append(q)
        csr.routing = len(routings)
        return csr

    monkeypatch.setattr(fv, "alloc_csr", lambda B, H, S, device, codes=False: Csr(B, H, S))
    monkeypatch.setattr(fv, "route", route)
    monkeypatch.setattr(fv, "sparse_attn", lambda q, k, v, csr, **kw: log.append(("sparse", csr.routing)))
    monkeypatch.setattr(fv, "dense_attn", lambda q, k, v, **kw: log.append(("dense",)))
    return log


def generation(layer, steps, calls):
    q = torch.zeros((1, 2, 100, 64))
    del calls[:]
    for step in steps:
        layer(q, q, q, step)
    return list(calls)


@pytest.mark.parametrize("steps,dense,every", [(16, 10, 8), (8, 5, 4), (5, 1, 4), (8, 2, 6), (50, 5, 4), (3, 2, 1),
                                               (4, 0, 4), (8, 0, 4), (5, 0, 4), (3, 0, 100)])
def test_every_generation_routes_afresh(calls, steps, dense, every):
    layer = fv.LazyRouter(fv.RouteConfig(), refresh_every=every, dense_steps=dense)
    routed = list(range(dense, steps, every))
    before = 0
    for _ in range(3):
        want = [("dense",)] * dense + [("sparse", before + 1 + (s - dense) // every) for s in range(dense, steps)]
        assert generation(layer, range(steps), calls) == want
        before += len(routed)
    assert layer.routed == before


def test_a_generation_that_ends_early_or_starts_late(calls):
    layer = fv.LazyRouter(fv.RouteConfig(), refresh_every=4, dense_steps=3)
    assert generation(layer, range(2), calls) == [("dense",)] * 2
    assert generation(layer, range(5), calls)[3:] == [("sparse", 1)] * 2
    assert generation(layer, range(2, 6), calls) == [("dense",)] + [("sparse", 2)] * 3
    assert generation(layer, range(4, 6), calls) == [("sparse", 3)] * 2


def test_two_calls_of_a_step_share_its_routing(calls):
    # with and without a condition, each step
    layer = fv.LazyRouter(fv.RouteConfig(), refresh_every=2, dense_steps=1)
    got = generation(layer, [0, 0, 1, 1, 2, 2, 3, 3], calls)
    assert got == [("dense",)] * 2 + [("sparse", 1)] * 4 + [("sparse", 2)] * 2
