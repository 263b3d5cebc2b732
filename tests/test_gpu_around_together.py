"""Routed attention, attention over all keys with its gradients, single tokens and the norm at once on four
streams: they share the SMs' tensor memory, and each gives the bits that it gives alone."""
import pytest
import torch

import block_sparse_top_fvattn_b200 as fv
from dense_cases import draw, run

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def test_every_kind_of_call_at_once():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn((1, 8, 3000, 128), generator=g).to(BF16).cuda() for _ in range(3))
    csrs = {}

    def routed():
        s = torch.cuda.current_stream()
        csrs[s] = fv.route(q, k, fv.RouteConfig(p=0.8), csr=csrs.get(s))
        return [fv.sparse_attn(q, k, v, csrs[s])]

    train = [draw(1, 6, 2, 900, 900, d, BF16, seed=d) for d in (64, 128)]
    few = draw(4, 16, 4, 1, 4000, 128, BF16, seed=3)
    x = torch.randn((2, 3000, 12, 128), generator=g).to(BF16).cuda()
    w = torch.ones(128, device="cuda")
    cfg = fv.AttnConfig(causal=True, softcap=30.0)
    kinds = [routed, lambda: list(run(train[0], cfg).values()), lambda: list(run(train[1], cfg).values()),
             lambda: list(run(few, cfg, grads=False).values()),
             lambda: list(fv.qk_norm_rope_bwd(q.expand(2, -1, -1, -1)[:, :, :3000].contiguous(),
                                              k.expand(2, -1, -1, -1)[:, :4].contiguous(), x[:, :, :8], x[:, :, 8:], w, w))]
    want = [f() for f in kinds]
    streams = [torch.cuda.Stream() for _ in kinds]
    torch.cuda.synchronize()
    for f, s in zip(kinds, streams):
        with torch.cuda.stream(s):
            f()                              # each stream's own routing buffers
    torch.cuda.synchronize()
    for _ in range(10):
        got = []
        for f, s in zip(kinds, streams):
            with torch.cuda.stream(s):
                got.append(f())
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(s, t) for s, t in zip(a, b))
