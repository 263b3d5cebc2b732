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
