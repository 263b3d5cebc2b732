"""A layer over several generations: each attends as a new layer would."""
import pytest
import torch

import block_sparse_top_fvattn_b200 as fv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fv.load()


@pytest.mark.parametrize("steps,dense,every", [(4, 2, 2), (3, 0, 4), (3, 1, 4)])
def test_a_second_generation_attends_as_a_new_layer(steps, dense, every):
    g = torch.Generator().manual_seed(0)
    used = fv.LazyRouter(fv.RouteConfig(p=0.5), refresh_every=every, dense_steps=dense)
    for _ in range(3):
        fresh = fv.LazyRouter(fv.RouteConfig(p=0.5), refresh_every=every, dense_steps=dense)
        for step in range(steps):
            q, k, v = (torch.randn((1, 2, 900, 64), generator=g).to(torch.bfloat16).cuda() for _ in range(3))
            assert torch.equal(used(q, k, v, step), fresh(q, k, v, step)), step


def test_a_layer_on_a_stream_beside_a_busy_one():
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn((1, 4, 1200, 64), generator=g).to(torch.bfloat16).cuda() for _ in range(3))
    plain = fv.LazyRouter(fv.RouteConfig(p=0.5), dense_steps=1)
    want = [plain(q, k, v, step) for step in range(3)]
    side, a = torch.cuda.Stream(), torch.randn((4096, 4096), device="cuda")
    layer = fv.LazyRouter(fv.RouteConfig(p=0.5), dense_steps=1)
    torch.cuda.synchronize()
    for step in range(3):
        for _ in range(20):
            a = a @ a * 1e-3
        for t in want:
            torch.empty_like(t).fill_(float("nan"))
        got = layer(q, k, v, step, stream=side)
        side.synchronize()
        torch.cuda.synchronize()
        assert torch.equal(got, want[step])
