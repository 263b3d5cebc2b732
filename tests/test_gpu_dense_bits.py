"""What must not matter does not reach a bit of attention over all keys: shared memory that earlier
kernels left, memory behind the valid keys, and padding tokens. A cap chooses a form of tanh by the
largest score in sight, so capped calls are the ones to look at."""
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


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def equal(a, b):
    for n in a:
        assert torch.equal(a[n], b[n]), f"{n}: {(a[n] != b[n]).sum().item()} of {a[n].numel()} differ"


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [3, 5, 12, 50])
@pytest.mark.parametrize("bias", [False, True])
def test_rows_of_a_tile_that_no_query_fills(d, G, bias):
    # G does not divide the tiles' rows: the last ones keep what the kernel before left in shared memory
    x = draw(1, G, 1, 150, 140, d, BF16, seed=1)
    cfg = fv.AttnConfig(softcap=30.0, slopes=torch.full((G,), 0.01, device="cuda") if bias else None)
    dirty_cfg = fv.AttnConfig(softcap=30.0, slopes=torch.full((6,), 0.01, device="cuda") if bias else None)
    got = []
    for size in (0.0, 1e3):
        # the same kernels, all rows of all SMs' tiles in use, queries of this size
        dirty = draw(1, 6, 6, 12800, 128, d, BF16, seed=2)
        dirty["q"] *= size
        dirty["dout"] *= size
        run(dirty, dirty_cfg)
        got.append(run(x, cfg))
    equal(*got)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("what", [1e4, -1e4, float("nan"), float("inf")])
@pytest.mark.parametrize("shape", [(2, 4, 2, 170, 300, 64), (2, 6, 2, 100, 260, 128), (2, 8, 2, 1, 1000, 128)])
def test_memory_behind_the_valid_keys(dtype, what, shape):
    x = draw(*shape, dtype, seed=3)
    Sk = shape[4]
    kv = (Sk - 13, Sk - 90)
    cfg = fv.AttnConfig(softcap=30.0, kv_len=i32(*kv), causal=shape[3] == 170)
    got = []
    for fill in (0.0, what):
        for b, n in enumerate(kv):
            x["k"][b, :, n:], x["v"][b, :, n:] = fill, fill
        got.append(run(x, cfg))
    equal(*got)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("what", [1e4, float("nan"), float("inf")])
@pytest.mark.parametrize("shape", [(1, 4, 2, 300, 300, 64), (1, 3, 1, 200, 200, 128)])
def test_padding_tokens(dtype, what, shape):
    x = draw(*shape, dtype, seed=4)
    S = shape[3]
    doc = torch.arange(S, dtype=torch.int32, device="cuda")[None] // 90
    doc[0, 33:50] = -1
    doc[0, 150:161] = -7
    doc[0, S - 21:] = -1
    pad = doc[0] < 0
    got = []
    for causal in (False, True):
        cfg = fv.AttnConfig(softcap=30.0, doc_q=doc, doc_k=doc, causal=causal)
        got.append([])
        for fill in (0.0, what):
            for n in x:
                x[n][:, :, pad] = fill
            got[-1].append(run(x, cfg))
    for a, b in got:
        equal(a, b)


def test_keys_that_an_order_or_another_document_hides():
    # finite, but far larger than what is in sight of the rows before them (whole warps of 16 queries: a
    # form is chosen for a warp)
    S, d = 256, 64
    x = draw(1, 4, 2, S, S, d, BF16, seed=5)
    doc = (torch.arange(S, dtype=torch.int32, device="cuda")[None] >= 128 + 32).int()
    for cfg, rows in ((fv.AttnConfig(softcap=30.0, causal=True), 176),
                      (fv.AttnConfig(softcap=30.0, doc_q=doc, doc_k=doc), 160)):
        got = []
        for size in (1.0, 1e3):
            y = {n: t.clone() for n, t in x.items()}
            y["k"][:, :, rows:] *= size
            o = run(y, cfg)
            got.append({n: o[n][:, :, :rows] for n in ("out", "lse", "dq")})
        equal(*got)
