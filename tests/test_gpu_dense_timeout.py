"""The failure path of the bounded waits in attention over all keys and its gradients, run on purpose without
a GPU fault: at a given step the loader of every CTA waits, with a short limit, on a barrier that
nothing completes, with the copies and products of the steps before in flight. Rows of a CTA that
stopped are NaN, others have their usual bits, the status says so, and the stream goes on."""
import pytest
import torch

import block_sparse_top_fvattn_b200 as fv
from block_sparse_top_fvattn_b200 import _lib
from dense_cases import draw, run

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fv.load()


def documents(S, length, pad):
    doc = torch.arange(S, dtype=torch.int32, device="cuda")[None] // length
    doc[0, S // 2:S // 2 + pad] = -1
    return doc


def config(shape, docs):
    if not docs:
        return fv.AttnConfig(softcap=30.0)
    doc = documents(shape[4], 150, 20)
    return fv.AttnConfig(softcap=30.0, doc_q=doc[:, -shape[3]:].contiguous(), doc_k=doc)


def nan_rows(t, usual):
    """Which rows are NaN throughout; the others have the usual bits."""
    gone = t.isnan().all(-1)
    assert torch.equal(t.isnan().any(-1), gone)
    assert torch.equal(t[~gone], usual[~gone])
    return gone


FORWARD = [   # shape, documents, steps that every CTA has, detail
    ((1, 16, 16, 1500, 400, 64), False, 7, 20),       # 64-key steps, one CTA per tile
    ((1, 16, 16, 1500, 400, 128), False, 7, 20),
    ((1, 2, 2, 300, 700, 128), False, 3, 20),         # the keys split over CTAs
    ((1, 8, 4, 700, 700, 64), True, 1, 20),           # documents, padding copied by hand
    ((2, 8, 2, 1, 3000, 128), False, 1, 520),         # few rows: clusters, and a join through memory
    ((1, 4, 1, 1, 500, 64), False, 1, 520),
    ((1, 8, 2, 3, 700, 64), True, 1, 520),
]


@pytest.mark.parametrize("shape,docs,least,detail", FORWARD)
@pytest.mark.parametrize("step,polls", [(0, 1), (0, 64), (1, 64), (2, 64), (3, 64), (5, 64)])
def test_forward_wait_runs_out(shape, docs, least, detail, step, polls):
    x = draw(*shape, BF16, seed=1)
    cfg = config(shape, docs)
    usual = run(x, cfg, grads=False)
    code, at, out, lse = fv.dense_attn_timeout_check(x["q"], x["k"], x["v"], cfg, step=step, polls=polls)
    gone = nan_rows(out, usual["out"])
    assert torch.equal(lse.isnan(), gone)
    if gone.any():
        assert (code, at) == (_lib.FVATTN_ERR_TIMEOUT, detail)
    else:
        assert step >= least and code == 0
    if step < least and not docs:
        assert gone.all()
    again = run(x, cfg, grads=False)                  # the stream and the context stay usable
    assert all(torch.equal(again[n], usual[n]) for n in usual)


BACKWARD = [   # shape, documents, the most steps of a CTA of dK and dV (of each cluster), steps of dQ
    ((1, 2, 1, 300, 256, 64), False, 5, 2),           # clusters of two CTAs: 10 steps of 32 queries
    ((1, 2, 1, 300, 256, 128), False, 5, 2),
    ((1, 3, 1, 700, 200, 128), False, 5, 2),          # clusters of eight: 34 steps of 21 queries
    ((1, 16, 4, 600, 4000, 64), False, 38, 32),       # one CTA per key tile
    ((1, 8, 4, 700, 700, 64), True, 0, 0),            # documents, padding copied by hand
]


@pytest.mark.parametrize("shape,docs,dkv_steps,dq_steps", BACKWARD)
@pytest.mark.parametrize("step,polls", [(0, 1), (0, 64), (1, 64), (2, 64), (4, 64), (7, 64), (1000, 64)])
def test_backward_wait_runs_out(shape, docs, dkv_steps, dq_steps, step, polls):
    x = draw(*shape, BF16, seed=2)
    cfg = config(shape, docs)
    usual = run(x, cfg, rest=False)
    code, at, dq, dk, dv = fv.dense_attn_bwd_timeout_check(x["dout"], x["q"], x["k"], x["v"], usual["out"], usual["lse"],
                                                           cfg, step=step, polls=polls)
    gone = {n: nan_rows(t, usual[n]) for n, t in (("dq", dq), ("dk", dk), ("dv", dv))}
    assert torch.equal(gone["dk"], gone["dv"])
    if step < dkv_steps:
        assert gone["dk"].all()
    if step < dq_steps:
        assert gone["dq"].all()
    any_gone = any(g.any() for g in gone.values())
    assert code == (_lib.FVATTN_ERR_TIMEOUT if any_gone else 0)
    if any_gone:
        assert at == (320 if gone["dk"].any() else 420)
    if step == 1000:
        assert not any_gone
    again = run(x, cfg, rest=False)
    assert all(torch.equal(again[n], usual[n]) for n in usual)


def test_timeout_checks_refuse_bad_arguments():
    x = draw(1, 2, 1, 20, 30, 64, BF16)
    got = run(x, fv.AttnConfig(), rest=False)
    f = {n: t.float() for n, t in x.items()}
    lse = got["lse"]
    for code, a, kw in ((_lib.FVATTN_ERR_INVALID, x, dict(polls=0)), (_lib.FVATTN_ERR_UNSUPPORTED, f, {})):
        with pytest.raises(fv.FvattnError) as e:
            fv.dense_attn_timeout_check(a["q"], a["k"], a["v"], **kw)
        assert e.value.code == code
        with pytest.raises(fv.FvattnError) as e:
            fv.dense_attn_bwd_timeout_check(a["dout"], a["q"], a["k"], a["v"], got["out"].to(a["q"].dtype), lse, **kw)
        assert e.value.code == code
