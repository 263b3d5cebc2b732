"""Calls on a given stream beside a busy current one, and inside a capture."""
import pytest
import torch

import block_sparse_top_fvattn_b200 as fv
from dense_cases import draw, run

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fv.load()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", [(2, 4, 2, 200, 200, 64), (2, 8, 2, 1, 2000, 128)])
def test_a_busy_current_stream_whose_temporaries_were_freed(dtype, shape):
    x = draw(*shape, dtype)
    cfg = fv.AttnConfig(softcap=30.0)
    lse = torch.empty(x["q"].shape[:3], device="cuda")

    def calls(**kw):
        o = fv.dense_attn(x["q"], x["k"], x["v"], cfg, lse=lse, **kw)
        return [o, *fv.dense_attn_bwd(x["dout"], x["q"], x["k"], x["v"], o, lse, cfg, **kw)]

    want = calls()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    a = torch.randn((4096, 4096), device="cuda")
    for _ in range(3):
        for _ in range(20):                 # some milliseconds of work
            a = a @ a * 1e-3
        # temporaries of the outputs' and the scratch's sizes, written behind that work and freed now
        for t in want:
            for _ in range(4):
                torch.empty_like(t).fill_(float("nan"))
        torch.empty(1 << 20, dtype=torch.uint8, device="cuda").fill_(255)
        got = calls(stream=side)            # does not wait for the current stream
        side.synchronize()
        copies = [t.clone() for t in got]
        torch.cuda.synchronize()
        assert all(torch.equal(c, w) for c, w in zip(copies, want))
        assert all(torch.equal(t, w) for t, w in zip(got, want))


def test_calls_on_a_stream_inside_a_capture():
    x = draw(2, 4, 2, 130, 170, 64, BF16)
    p = {n: torch.randn((2, 130, h, 64), device="cuda").to(BF16) for n, h in (("q", 4), ("k", 2))}
    w = [torch.randn(64, device="cuda") for _ in range(2)]
    g = {"q": torch.randn((2, 4, 130, 64), device="cuda").to(BF16), "k": torch.randn((2, 2, 130, 64), device="cuda").to(BF16)}
    cfg = fv.AttnConfig(softcap=30.0, causal=True)

    def calls(**kw):
        got = [*run(x, cfg, **kw).values(), *fv.qk_norm_rope(p["q"], p["k"], *w, **kw)]
        return got + list(fv.qk_norm_rope_bwd(g["q"], g["k"], p["q"], p["k"], *w, **kw))

    calls()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = calls(stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for t in (*x.values(), *p.values(), *g.values()):
        t.mul_(-0.5)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, calls()))


def test_two_graphs_with_scratch_of_their_own_replayed_at_once():
    cfg = fv.AttnConfig(softcap=30.0)
    xs = [draw(2, 8, 2, 1, 5000, 128, BF16, seed=s) for s in (1, 2)]
    want = [run(x, cfg) for x in xs]
    graphs, got = [], []
    for x in xs:
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(run(x, cfg))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(a[n], b[n]) for n in a)
