"""Attention over all keys with capped, biased and masked scores, and its gradients, against the fp64
oracle within bounds derived from the kernels' roundings (dense_cases)."""
import numpy as np
import pytest
import torch

import block_sparse_top_fvattn_b200 as fv
from dense_cases import bounds, compare, draw, f64, reference, run

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fv.load()


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def slopes(H):
    return (2.0 ** -torch.arange(1, H + 1, dtype=torch.float32)).cuda()


def documents(B, S, mean, pad=0, seed=0):
    """Ascending document numbers with lengths around `mean`, the last `pad` tokens padding."""
    rng = np.random.default_rng(seed)
    d = np.cumsum(rng.random((B, S)) < 1.0 / mean, axis=1).astype(np.int32)
    if pad:
        d[:, S - pad:] = -1
    return torch.from_numpy(d).cuda()


def check(shape, dtype, cfg, seed=0, spread=1.0, grads=True, scale=None, x=None, **kw):
    x = x or draw(*shape, dtype, seed, spread)
    got = run(x, cfg, grads=grads, **kw, **({"scale": scale} if scale else {}))
    r = reference(x, cfg, scale=scale, grads=grads)
    compare(got, r, bounds(r, cfg, dtype))
    return x, got, r


SHAPES = [   # B, Hq, Hkv, Sq, Sk, d
    (1, 1, 1, 1, 1, 64), (1, 1, 1, 1, 1, 128), (2, 2, 2, 64, 64, 64), (1, 2, 2, 63, 65, 128), (1, 2, 1, 129, 127, 64),
    (2, 4, 2, 128, 128, 128), (1, 3, 1, 200, 333, 64), (1, 15, 3, 101, 140, 128), (1, 16, 1, 70, 300, 64),
    (1, 64, 1, 3, 77, 128), (1, 50, 1, 5, 66, 64), (3, 2, 2, 257, 1, 64), (1, 1, 1, 300, 700, 128),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("causal", [False, True])
def test_sizes(shape, dtype, causal):
    check(shape, dtype, fv.AttnConfig(causal=causal), seed=1)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap", [0.5, 5.0, 50.0, 200.0])
def test_softcap(dtype, d, cap):
    check((1, 4, 2, 150, 190, d), dtype, fv.AttnConfig(softcap=cap, causal=cap == 5.0), spread=3.0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("cap", [0.0, 10.0])
def test_distance_bias(dtype, causal, cap):
    check((2, 6, 2, 140, 200, 64), dtype, fv.AttnConfig(slopes=slopes(6), causal=causal, softcap=cap))
    # a slope that favours far keys
    check((1, 2, 2, 70, 90, 128), dtype, fv.AttnConfig(slopes=-slopes(2), causal=causal, softcap=cap))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prefix_and_lengths(dtype):
    # prefixes below, inside, beyond the sequence and negative; lengths 0, 1, inside, beyond
    cfg = fv.AttnConfig(causal=True, prefix_len=i32(0, 30, 400, -5), kv_len=i32(0, 1, 131, 400))
    _, got, _ = check((4, 4, 2, 150, 150, 64), dtype, cfg)
    assert (got["out"][0] == 0).all() and (got["lse"][0] == -np.inf).all() and (got["dq"][0] == 0).all()
    cfg = fv.AttnConfig(kv_len=i32(-3, 64, 65, 99), q_start=i32(7, 7, 7, 7))
    check((4, 2, 2, 33, 99, 128), dtype, cfg)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("start", [-40, -1000, 0, 13, 5000, -2**31, 2**31 - 1])
def test_query_positions(dtype, start):
    # negative positions leave the first rows empty, large ones see everything
    check((2, 2, 1, 90, 110, 64), dtype, fv.AttnConfig(causal=True, q_start=i32(start, 3)))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("mean", [3, 40, 150])
def test_documents(dtype, causal, mean):
    doc = documents(2, 333, mean, pad=17)
    check((2, 4, 2, 333, 333, 64), dtype, fv.AttnConfig(causal=causal, doc_q=doc, doc_k=doc, softcap=20.0))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_documents_in_any_order(dtype):
    g = torch.Generator().manual_seed(3)
    dq = torch.randint(-1, 4, (2, 200), generator=g, dtype=torch.int32).cuda()
    dk = torch.randint(-1, 4, (2, 310), generator=g, dtype=torch.int32).cuda()
    dk[1] = 7                                     # no query of the second sequence sees anything
    _, got, _ = check((2, 3, 1, 200, 310, 128), dtype, fv.AttnConfig(doc_q=dq, doc_k=dk))
    assert (got["out"][1] == 0).all() and (got["dk"][1] == 0).all() and (got["dv"][1] == 0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), torch.finfo(torch.bfloat16).min])
def test_masked_memory_may_hold_anything(dtype, what):
    # behind the valid keys, and in padding tokens
    x = draw(2, 2, 1, 150, 200, 64, dtype)
    x["k"][0, :, 77:], x["v"][0, :, 77:] = what, what
    x["k"][1, :, :], x["v"][1, :, :] = what, what
    check(None, dtype, fv.AttnConfig(kv_len=i32(77, 0)), x=x)
    x = draw(1, 4, 2, 170, 170, 128, dtype)
    doc = documents(1, 170, 50)
    doc[0, 40:60], doc[0, 128:140] = -1, -5
    for n in ("q", "k", "v", "dout"):
        x[n][:, :, (doc[0] < 0).cpu()] = what
    check(None, dtype, fv.AttnConfig(doc_q=doc, doc_k=doc, causal=True), x=x)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", [(1, 1, 1, 1, 5000, 128), (2, 8, 2, 1, 3001, 64), (1, 32, 8, 1, 4096, 128),
                                   (3, 4, 4, 2, 777, 128), (1, 16, 1, 7, 2050, 64), (5, 40, 8, 1, 129, 128)])
def test_few_queries_over_many_keys(dtype, shape):
    B, Hq, _, Sq, Sk, _ = shape
    kv = [max(0, Sk - 611 * b) for b in range(B)]
    kv[-1] = 0 if B > 1 else Sk
    cfg = fv.AttnConfig(causal=True, kv_len=i32(*kv), q_start=i32(*[max(0, n - Sq) for n in kv]), softcap=30.0,
                        slopes=slopes(Hq))
    check(shape, dtype, cfg, spread=2.0)
    check(shape, dtype, fv.AttnConfig(), spread=2.0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap", [0.0, 25.0])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("docs", [False, True])
def test_all_together(dtype, d, cap, bias, docs):
    # every combination of the kernels' variants, for whole sequences and for one to eight queries (up to
    # 16, 24 and 32 rows of a shared key head)
    for B, Hq, Hkv, Sq, Sk in ((2, 4, 2, 190, 190), (2, 6, 2, 1, 300), (1, 16, 1, 1, 700), (2, 8, 2, 4, 333),
                               (1, 8, 1, 3, 500), (1, 4, 1, 8, 270)):
        doc_k = documents(B, Sk, 60, pad=9, seed=4) if docs else None
        doc_q = doc_k[:, Sk - Sq:].contiguous() if docs else None
        if docs and Sq > 1:
            doc_q[:, -1] = doc_q[:, 0]
        cfg = fv.AttnConfig(causal=True, softcap=cap, slopes=slopes(Hq) if bias else None, doc_q=doc_q, doc_k=doc_k,
                            prefix_len=i32(*[11 * b for b in range(B)]), kv_len=i32(*[Sk - 5 * b for b in range(B)]))
        check((B, Hq, Hkv, Sq, Sk, d), dtype, cfg, seed=Sq, spread=2.0)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strides(dtype):
    # slices of one [B, S, H, d] projection, a place in a longer cache, transposed outputs
    B, Hq, Hkv, S, d = 2, 4, 2, 140, 64
    g = torch.Generator().manual_seed(0)
    w = torch.randn((B, S, Hq + 2 * Hkv, d), generator=g).to(dtype).cuda()
    q = w[:, :, :Hq].transpose(1, 2)
    cache = torch.full((2, B, Hkv, S + 77, d), float("nan"), dtype=dtype, device="cuda")
    cache[0, :, :, :S], cache[1, :, :, :S] = w[:, :, Hq:Hq + Hkv].transpose(1, 2), w[:, :, Hq + Hkv:].transpose(1, 2)
    k, v = cache[0, :, :, :S], cache[1, :, :, :S]
    dout = torch.randn((B, S, Hq, d), generator=g).to(dtype).cuda().transpose(1, 2)
    x = {"q": q, "k": k, "v": v, "dout": dout}
    cfg = fv.AttnConfig(causal=True)
    lse = torch.empty((B, Hq, S), device="cuda")
    out = torch.empty((B, S, Hq, d), dtype=dtype, device="cuda").transpose(1, 2)
    rest = torch.empty((B, S, Hq, d), dtype=dtype, device="cuda").transpose(1, 2) if dtype == BF16 else None
    dw = torch.full_like(w, 7.0)
    got = {"out": fv.dense_attn(q, k, v, cfg, out=out, rest=rest, lse=lse), "lse": lse}
    got["dq"], got["dk"], got["dv"] = fv.dense_attn_bwd(
        dout, q, k, v, out, lse, cfg, rest=rest, dq=dw[:, :, :Hq].transpose(1, 2),
        dk=dw[:, :, Hq:Hq + Hkv].transpose(1, 2), dv=dw[:, :, Hq + Hkv:].transpose(1, 2))
    r = reference(x, cfg)
    compare(got, r, bounds(r, cfg, dtype))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_writes_only_its_outputs(dtype):
    # every output lies in a larger buffer; what surrounds it keeps its values
    B, Hq, Hkv, Sq, Sk, d = 2, 6, 2, 75, 131, 64
    x = draw(B, Hq, Hkv, Sq, Sk, d, dtype)
    cfg = fv.AttnConfig(causal=True)

    def inside(H, S):
        big = torch.full((B + 1, H + 1, S + 3, d), 5.0, dtype=dtype, device="cuda")
        return big, big[:B, :H, 1:S + 1]

    (bo, out), (bq, dq), (bk, dk), (bv, dv) = inside(Hq, Sq), inside(Hq, Sq), inside(Hkv, Sk), inside(Hkv, Sk)
    lse = torch.empty((B, Hq, Sq), device="cuda")
    fv.dense_attn(x["q"], x["k"], x["v"], cfg, out=out, lse=lse)
    fv.dense_attn_bwd(x["dout"], x["q"], x["k"], x["v"], out, lse, cfg, dq=dq, dk=dk, dv=dv)
    r = reference(x, cfg)
    compare({"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}, r, bounds(r, cfg, dtype, rest=False))
    for big, part in ((bo, out), (bq, dq), (bk, dk), (bv, dv)):
        part.fill_(5.0)
        assert (big == 5.0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_equal_calls_give_equal_bits(dtype):
    x = draw(2, 8, 2, 300, 420, 64, dtype)
    cfg = fv.AttnConfig(softcap=15.0, slopes=slopes(8))
    a, b = run(x, cfg), run(x, cfg)
    assert all(torch.equal(a[n], b[n]) for n in a)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scale_and_large_scores(dtype):
    check((1, 2, 2, 100, 130, 64), dtype, fv.AttnConfig(), scale=0.7, spread=6.0)
    # scores whose exponential overflows fp32 without the running maximum, ascending along the keys
    x = draw(1, 1, 1, 70, 300, 64, dtype, spread=0.1)
    x["k"] *= torch.linspace(0.1, 30, 300, device="cuda")[:, None].to(dtype)
    x["q"] += 1
    check(None, dtype, fv.AttnConfig(), x=x, scale=1.0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", [(2, 4, 2, 200, 200, 64), (2, 8, 2, 1, 2000, 128)])
def test_captured_and_replayed_on_another_stream(dtype, shape):
    B, _, _, Sq, Sk, _ = shape
    x = draw(*shape, dtype)
    kv, start = i32(*[Sk] * B), i32(*[Sk - Sq] * B)
    cfg = fv.AttnConfig(causal=True, kv_len=kv, q_start=start, softcap=30.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(x, cfg)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = run(x, cfg)
    for seed, n in ((5, Sk), (6, Sk - 3)):
        new = draw(*shape, dtype, seed=seed)
        for name in x:
            x[name].copy_(new[name])
        kv.fill_(n)
        start.fill_(n - Sq)
        g.replay()
        torch.cuda.synchronize()
        r = reference(x, cfg)
        compare(got, r, bounds(r, cfg, dtype))
    # the stream argument, with inputs made on the current stream
    direct = run(x, cfg)
    side.wait_stream(torch.cuda.current_stream())
    other = run(x, cfg, stream=side)
    side.synchronize()
    assert all(torch.equal(direct[n], other[n]) for n in direct)


def test_two_calls_at_once_on_two_streams():
    shape = (2, 8, 2, 1, 3000, 128)
    xs = [draw(*shape, BF16, seed=s) for s in (1, 2)]
    cfg = fv.AttnConfig(softcap=30.0)
    want = [run(x, cfg, grads=False) for x in xs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        got = []
        for x, s in zip(xs, streams):
            with torch.cuda.stream(s):
                got.append(run(x, cfg, grads=False))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(a[n], b[n]) for n in a)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cap", [30.0, 50.0, 50.5, 100.0])
def test_saturated_caps_and_large_values(dtype, cap):
    # every score at the cap or at its negative (scores of 25 times the cap: tanh is 1 to fp32), with and
    # without a running maximum, and values whose sums times e^50 are 2^118
    Sq, Sk, d = 130, 300, 64
    x = draw(1, 2, 1, Sq, Sk, d, dtype)
    sign = torch.ones(Sq, device="cuda")
    sign[::2] = -1
    x["q"] = (sign[:, None] * torch.ones(1, 2, Sq, d, device="cuda")).to(dtype)
    x["k"] = torch.ones(1, 1, Sk, d, device="cuda").to(dtype)
    x["v"] = x["v"] * 2.0 ** 34
    cfg = fv.AttnConfig(softcap=cap)
    got = run(x, cfg, grads=False, scale=25.0 * cap / d)
    # equal scores: out is the mean of the values, lse the score plus log Sk
    v = f64(x["v"])
    u = 2.0 ** -8 if dtype == BF16 else 2.0 ** -24
    mean, size = v.mean(axis=2, keepdims=True), np.abs(v).mean(axis=2, keepdims=True)
    # the weight's rounding and the sum of Sk terms on mean |v|, the rounding of out
    tol = (u + (Sk + 8) * 2 * 2.0 ** -24) * size + u * np.abs(mean)
    assert (np.abs(f64(got["out"]) - mean) <= tol).all()
    want = np.where(np.arange(Sq) % 2 == 0, -cap, cap) + np.log(Sk)
    assert (np.abs(f64(got["lse"]) - want) <= 8 * 2.0 ** -24 * (2 * cap + 8) + (Sk + 8) * 2.0 ** -23).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gradients_at_once_on_two_streams(dtype):
    shape = (1, 4, 2, 260, 300, 64)
    xs = [draw(*shape, dtype, seed=s) for s in (1, 2)]
    doc = [documents(1, n, 70, seed=3) for n in (260, 300)]
    cfg = fv.AttnConfig(softcap=30.0, doc_q=doc[0], doc_k=doc[1])
    want = [run(x, cfg) for x in xs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):
        got = []
        for x, s in zip(xs, streams):
            with torch.cuda.stream(s):
                got.append(run(x, cfg))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(a[n], b[n]) for n in a)


def test_long_cache_offsets_past_32_bits():
    # one key head of a cache of 2^25 + 70 tokens: byte and element offsets beyond 2^32
    S, d = (1 << 25) + 70, 128
    k = torch.zeros((1, 1, S, d), dtype=BF16, device="cuda")
    v = torch.zeros((1, 1, S, d), dtype=BF16, device="cuda")
    q = torch.ones((1, 1, 1, d), dtype=BF16, device="cuda")
    k[0, 0, -3:] = 4.0                            # score 4 * 128 / sqrt(128) = 45 against 0
    v[0, 0, -3:, :] = torch.tensor([1.0, 2.0, 6.0], dtype=BF16, device="cuda")[:, None]
    out = fv.dense_attn(q, k, v)
    # weights: three keys of e^45.25 against 2^25 of 1: the rest has 3e-13 of the mass
    np.testing.assert_allclose(f64(out), 3.0, rtol=2.0 ** -8)
