"""Cases, plain forms and 64-bit values of two operators around an attention layer:

norm   per-head RMS norm of the projected queries and keys with the position rotation in the
       same pass, from [B, S, H, d] to the [B, H, S, d] of the attention (fv.qk_norm_rope), and
       its gradients (fv.qk_norm_rope_bwd)
attn   exact attention over all keys whose scores may be capped by a tanh, biased by distance,
       and masked by length, order, prefix and document (fv.dense_attn), and its gradients
       (fv.dense_attn_bwd)

With `own` false, run() computes the plain form in elementary torch operations in 32 bits; with
`own` true it calls the library.
"""
import math
import random

import torch

own = False

EPS = 1e-6
THETA = 10000.0


def _fv():
    import block_sparse_top_fvattn_b200 as fv
    return fv


# ---------------------------------------------------------------------------------- the cases

def _norm(name, B, S, Hq, Hkv, d, *, dtype="bf16", rot=None, inter=True, far=0, train=False):
    return {"name": name, "op": "norm", "B": B, "S": S, "Hq": Hq, "Hkv": Hkv, "d": d, "dtype": dtype,
            "rot": d if rot is None else rot, "inter": inter, "far": far, "train": train}


def _attn(name, B, Sq, Sk, Hq, Hkv, d, *, dtype="bf16", cap=0.0, bias=False, causal=False, prefix=0, ragged=0,
          doc=0, train=False):
    return {"name": name, "op": "attn", "B": B, "Sq": Sq, "Sk": Sk, "Hq": Hq, "Hkv": Hkv, "d": d, "dtype": dtype,
            "cap": cap, "bias": bias, "causal": causal, "prefix": prefix, "ragged": ragged, "doc": doc,
            "train": train}


def listed():
    return [
        # one new token for each of 16 requests, at far positions: the smallest call, latency only
        _norm("norm-decode", 16, 1, 32, 8, 128, far=30000),
        # the 12-head layer of 8192 tokens, every dimension rotated in adjacent pairs
        _norm("norm-layer", 1, 8192, 12, 12, 128),
        # the 40-head layer of 21 frames of 1560 tokens: the largest tensors
        _norm("norm-large", 1, 32760, 40, 40, 128),
        # a training step's pass and its gradients, shared key heads, half-split pairs, part of the head rotated
        _norm("norm-train", 2, 4099, 16, 4, 64, rot=32, inter=False, train=True),
        # one new token for each of 4 requests with short caches: latency
        _attn("attn-decode-short", 4, 1, 1000, 8, 2, 128, ragged=300, causal=True, bias=True),
        # one new token for each of 8 requests with long caches of unequal length, capped scores
        _attn("attn-decode-long", 8, 1, 32760, 32, 8, 128, ragged=2047, causal=True, cap=50.0),
        # a batch of prompts whose first tokens are seen both ways, capped scores
        _attn("attn-prefix", 2, 2047, 2047, 16, 4, 128, causal=True, prefix=300, cap=30.0),
        # clips packed one after the other, each attending to itself only: a long sequence of documents
        _attn("attn-packed", 1, 16380, 16380, 6, 6, 128, doc=1560),
        # queries of one clip over padded conditioning tokens, biased by distance
        _attn("attn-cross", 3, 4099, 517, 12, 12, 64, ragged=100, bias=True),
        # the 32-bit path on the two-head layer of 1024 tokens
        _attn("attn-f32", 1, 1024, 1024, 2, 2, 64, dtype="f32", causal=True, cap=20.0),
        # a training step on packed documents with shared key heads and capped scores, odd sizes
        _attn("attn-train-packed", 2, 1999, 1999, 8, 2, 64, doc=450, causal=True, cap=30.0, train=True),
        # a training step of the 12-head layer of 8192 tokens, the first frame seen both ways
        _attn("attn-train-layer", 1, 8192, 8192, 12, 12, 128, causal=True, prefix=1024, train=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    heads = rng.choice([(2, 2), (8, 2), (12, 12), (12, 4), (16, 4), (16, 1), (15, 5), (40, 40), (32, 8)])
    d = rng.choice([64, 128])
    f32 = rng.random() < 0.15
    if rng.random() < 0.4:
        # at most the tokens of the largest listed case over its 40 + 40 heads, about 2.6 million rows
        rows = _log(rng, 512, 2600000)
        train = rng.random() < 0.4
        B = rng.choice([1, 1, 2, 3, 16])
        S = max(1, rows // (2 if train else 1) // (2 if f32 else 1) // (sum(heads) * B))
        rot = rng.choice([d, d, d // 2, 16 * rng.randint(1, d // 16)])
        c = _norm("", B, S, heads[0], heads[1], d, dtype="f32" if f32 else "bf16", rot=rot,
                  inter=rng.random() < 0.5, far=rng.choice([0, 0, _log(rng, 100, 30000)]), train=train)
    elif rng.random() < 0.35:
        # single new tokens (or a few of them): up to the cache bytes of the longest listed case
        B = rng.choice([1, 2, 4, 8, 13])
        Sk = _log(rng, 64, min(60000, 8 * 32760 * 8 // (B * heads[1]) * (128 // d)))
        if f32:
            Sk = max(1, Sk // 8)
        c = _attn("", B, rng.choice([1, 1, 1, 2, 4, 7]), max(Sk, 8), heads[0], heads[1], d,
                  dtype="f32" if f32 else "bf16",
                  cap=rng.choice([0.0, 0.0, 30.0]), bias=rng.random() < 0.3, causal=True,
                  ragged=rng.choice([0, max(1, Sk // 9)]))
    else:
        # whole sequences: at most the pairs of the largest listed case
        B = rng.choice([1, 1, 2, 3])
        train = rng.random() < 0.5
        most = math.sqrt(12 * 8192 * 8192 / (1 if train else 0.6) / (B * heads[0])) / (4 if f32 else 1)
        Sq = _log(rng, 64, min(most, 16380))
        Sk = Sq if rng.random() < 0.75 else _log(rng, 64, min(most, 8192))
        same = Sq == Sk
        causal = same and rng.random() < 0.6
        c = _attn("", B, Sq, Sk, heads[0], heads[1], d, dtype="f32" if f32 else "bf16",
                  cap=rng.choice([0.0, 0.0, 20.0, 50.0]), bias=rng.random() < 0.25, causal=causal,
                  prefix=Sq // 5 if causal and rng.random() < 0.4 else 0,
                  ragged=Sk // 7 if rng.random() < 0.3 else 0,
                  doc=max(8, Sq // rng.choice([3, 8, 20])) if same and rng.random() < 0.35 else 0, train=train)
    del c["name"]
    return c


# ---------------------------------------------------------------------------- what a case holds

def _kv_lens(case):
    """Valid keys of each sequence: unequal by about `ragged` from one to the next, at least one."""
    return [max(1, case["Sk"] - b * case["ragged"]) for b in range(case["B"])]


def _q_starts(case):
    """Position of the first query: a new token follows its cache; a whole sequence starts at 0."""
    if case["Sq"] == case["Sk"]:
        return [0] * case["B"]
    return [max(0, n - case["Sq"]) for n in _kv_lens(case)] if case["causal"] else [0] * case["B"]


def _prefix_lens(case):
    return [max(1, case["prefix"] - 37 * b) for b in range(case["B"])]


def _documents(case):
    """Document lengths of each sequence, from about a third of `doc` to about twice it."""
    rng = random.Random(case["doc"] * 1000003 + case["Sk"])
    out = []
    for _ in range(case["B"]):
        lens, left = [], case["Sk"]
        while left > 0:
            n = min(left, max(1, int(case["doc"] * rng.uniform(0.35, 1.8))))
            lens.append(n)
            left -= n
        out.append(lens)
    return out


def _pairs(case):
    """Visible (query, key) pairs of one head, over the batch."""
    total = 0
    kv, start = _kv_lens(case), _q_starts(case)
    for b in range(case["B"]):
        n, p0 = kv[b], start[b]
        pre = _prefix_lens(case)[b] if case["prefix"] else 0
        if case["doc"]:
            at = 0
            for length in _documents(case)[b]:
                for i in range(at, at + length):
                    hi = min(n, at + length, max(i + 1, pre)) if case["causal"] else min(n, at + length)
                    total += max(0, hi - at)
                at += length
        elif case["causal"]:
            for i in range(case["Sq"]):
                total += min(n, max(p0 + i + 1, pre))
        else:
            total += n * case["Sq"]
    return total


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    d = case["d"]
    if case["op"] == "norm":
        n = case["B"] * case["S"] * (case["Hq"] + case["Hkv"]) * d
        tokens = case["B"] * case["S"] if case["far"] else case["S"]
        table = tokens * case["rot"] * 4
        small = 2 * d * 4 + (case["B"] * case["S"] * 4 if case["far"] else 0)
        if not case["train"]:
            return {"bytes": 2 * n * e + table + small, "flops": 10 * n}
        # forward: x in, y out; backward: x and dy in, dx out
        return {"bytes": 5 * n * e + table + 2 * small, "flops": 30 * n}
    q = case["B"] * case["Hq"] * case["Sq"] * d * e
    kv = sum(_kv_lens(case)) * case["Hkv"] * d * e
    rows = case["B"] * case["Hq"] * case["Sq"] * 4
    pairs = _pairs(case) * case["Hq"]
    if not case["train"]:
        return {"bytes": 2 * q + 2 * kv + rows, "flops": 4 * d * pairs}
    # forward: q, k, v in, out and its row sums out; backward: dout in, dq, dk, dv out
    return {"bytes": 4 * q + 4 * kv + rows, "flops": 14 * d * pairs}


# -------------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _table(rows, rot):
    """cos and sin of position * theta^(-2i/rot), the angles in 64 bits, kept in 32."""
    inv = THETA ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * inv[None, :]
    return a.cos().float(), a.sin().float()


def prepare(case, seed):
    g = _gen(seed)
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    B, Hq, Hkv, d = case["B"], case["Hq"], case["Hkv"], case["d"]

    def normal(*shape, dtype=dt):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)

    if case["op"] == "norm":
        S, far = case["S"], case["far"]
        # queries and keys are slices of one projection's output, as a fused projection leaves them
        x = normal(B, S, Hq + 2 * Hkv, d)
        st = {"case": case, "q": x[:, :, :Hq], "k": x[:, :, Hq:Hq + Hkv],
              "wq": 1 + 0.2 * normal(d, dtype=torch.float32), "wk": 1 + 0.2 * normal(d, dtype=torch.float32)}
        st["cos"], st["sin"] = _table(far + S, case["rot"])
        st["pos"] = None
        if far:
            first = torch.randint(0, far + 1, (B, 1), generator=g, device="cuda", dtype=torch.int32)
            st["pos"] = (first + torch.arange(S, device="cuda", dtype=torch.int32)[None, :]).contiguous()
        if case["train"]:
            st["gq"], st["gk"] = normal(B, Hq, S, d), normal(B, Hkv, S, d)
        return st
    Sq, Sk = case["Sq"], case["Sk"]
    # scores of standard deviation about 2: some keys matter more than others
    st = {"case": case, "q": 2 * normal(B, Hq, Sq, d), "k": normal(B, Hkv, Sk, d), "v": normal(B, Hkv, Sk, d)}

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    st["kv_len"] = i32(_kv_lens(case)) if case["ragged"] else None
    st["q_start"] = i32(_q_starts(case)) if Sq != Sk else None
    st["prefix"] = i32(_prefix_lens(case)) if case["prefix"] else None
    st["doc"] = None
    if case["doc"]:
        st["doc"] = torch.stack([torch.repeat_interleave(torch.arange(len(n), dtype=torch.int32), torch.tensor(n))
                                 for n in _documents(case)]).cuda().contiguous()
    st["slopes"] = None
    if case["bias"]:
        st["slopes"] = 2.0 ** (-8.0 * torch.arange(1, Hq + 1, device="cuda", dtype=torch.float32) / Hq)
    if case["train"]:
        st["g"] = normal(B, Hq, Sq, d)
    return st


# --------------------------------------------------------------------------------- plain forms

def _pair_halves(x, rot, inter):
    return (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])


def _rotated(x, c, s, rot, inter):
    a, b = _pair_halves(x, rot, inter)
    a, b = a * c - b * s, a * s + b * c
    turned = torch.stack([a, b], -1).flatten(-2) if inter else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _angles(st):
    S = st["case"]["S"]
    if st["pos"] is None:
        return st["cos"][:S, None], st["sin"][:S, None]
    at = st["pos"].long()
    return st["cos"][at][:, :, None], st["sin"][at][:, :, None]


def _plain_norm(st):
    case = st["case"]
    rot, inter = case["rot"], case["inter"]
    c, s = _angles(st)

    def forward(x, w):
        x = x.float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        return _rotated(x * r * w, c, s, rot, inter).transpose(1, 2).contiguous()

    def backward(g, x, w):
        g = _rotated(g.float().transpose(1, 2), c, -s, rot, inter)
        x = x.float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        dw = (g * x * r).sum((0, 1, 2))
        gw = g * w
        return r * gw - x * r ** 3 * (gw * x).mean(-1, keepdim=True), dw

    dt = st["q"].dtype
    out = {"q": forward(st["q"], st["wq"]).to(dt), "k": forward(st["k"], st["wk"]).to(dt)}
    if case["train"]:
        dq, dwq = backward(st["gq"], st["q"], st["wq"])
        dk, dwk = backward(st["gk"], st["k"], st["wk"])
        out.update(dq=dq.to(dt), dk=dk.to(dt), dwq=dwq, dwk=dwk)
    return out


def _visible(st):
    """Bool [B or 1, 1, Sq, Sk], or None where every pair is visible."""
    case = st["case"]
    Sq, Sk = case["Sq"], case["Sk"]
    j = torch.arange(Sk, device="cuda")[None, None, None, :]
    p = torch.arange(Sq, device="cuda")[None, None, :, None]
    if st["q_start"] is not None:
        p = p + st["q_start"][:, None, None, None]
    see = None
    if case["causal"]:
        see = j <= p
        if st["prefix"] is not None:
            see = see | (j < st["prefix"][:, None, None, None])
    if st["kv_len"] is not None:
        short = j < st["kv_len"][:, None, None, None]
        see = short if see is None else see & short
    if st["doc"] is not None:
        mine = st["doc"][:, None, :, None] == st["doc"][:, None, None, :]
        see = mine if see is None else see & mine
    return see, (p - j).abs()


def _plain_attn(st):
    case = st["case"]
    dt = st["q"].dtype
    G = case["Hq"] // case["Hkv"]
    q, k, v = st["q"].float(), st["k"].float(), st["v"].float()
    B, _, Sk, d = k.shape
    Sq = case["Sq"]

    def grouped(x):                     # [B, Hq, Sq, n] as the rows of its shared key head
        return x.reshape(B, case["Hkv"], G * Sq, x.shape[-1])

    scale = 1 / math.sqrt(d)
    x = (grouped(q) @ k.transpose(-1, -2)).view(B, case["Hq"], Sq, Sk) * scale
    if case["cap"]:
        t = torch.tanh(x / case["cap"])
        x = t * case["cap"]
    see, far = _visible(st)
    if st["slopes"] is not None:
        x = x - st["slopes"][None, :, None, None] * far
    if see is not None:
        x = torch.where(see, x, -torch.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, 0.0)
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True)
    p = e / torch.where(total > 0, total, 1.0)
    lse = (top + torch.log(total)).squeeze(-1)
    o = (grouped(p) @ v).view(B, case["Hq"], Sq, d)
    out = {"out": o.to(dt), "lse": lse}
    if case["train"]:
        g = st["g"].float()
        dv = grouped(p).transpose(-1, -2) @ grouped(g)
        dp = (grouped(g) @ v.transpose(-1, -2)).view_as(p)
        ds = p * (dp - (p * dp).sum(-1, keepdim=True))
        if case["cap"]:
            ds = ds * (1 - t * t)
        ds = ds * scale
        dq = (grouped(ds) @ k).view_as(q)
        dk = grouped(ds).transpose(-1, -2) @ grouped(q)
        out.update(dq=dq.to(dt), dk=dk.to(dt), dv=dv.to(dt))
    return out


# ------------------------------------------------------------------------- the library's calls

def _own_norm(st):
    fv, case = _fv(), st["case"]
    opt = dict(positions=st["pos"], interleaved=case["inter"], eps=EPS)
    q, k = fv.qk_norm_rope(st["q"], st["k"], st["wq"], st["wk"], st["cos"], st["sin"], **opt)
    out = {"q": q, "k": k}
    if case["train"]:
        dq, dk, dwq, dwk = fv.qk_norm_rope_bwd(st["gq"], st["gk"], st["q"], st["k"], st["wq"], st["wk"], st["cos"],
                                               st["sin"], **opt)
        out.update(dq=dq, dk=dk, dwq=dwq, dwk=dwk)
    return out


def _own_attn(st):
    fv, case = _fv(), st["case"]
    cfg = fv.AttnConfig(softcap=case["cap"], causal=case["causal"], slopes=st["slopes"], q_start=st["q_start"],
                        prefix_len=st["prefix"], kv_len=st["kv_len"], doc_q=st["doc"], doc_k=st["doc"])
    q = st["q"]
    lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
    if not case["train"]:
        return {"out": fv.dense_attn(q, st["k"], st["v"], cfg, lse=lse), "lse": lse}
    # a training step also keeps what the rounding of the output to bf16 leaves, for the gradients
    rest = torch.empty_like(q) if q.dtype == torch.bfloat16 else None
    o = fv.dense_attn(q, st["k"], st["v"], cfg, lse=lse, rest=rest)
    dq, dk, dv = fv.dense_attn_bwd(st["g"], q, st["k"], st["v"], o, lse, cfg, rest=rest)
    return {"out": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def run(state):
    if state["case"]["op"] == "norm":
        return _own_norm(state) if own else _plain_norm(state)
    return _own_attn(state) if own else _plain_attn(state)


# --------------------------------------------------------------------------------- 64-bit values

def _exact_norm(case, st):
    rot, inter, S, B = case["rot"], case["inter"], case["S"], case["B"]
    pos = torch.arange(S, device="cuda").expand(B, S) if st["pos"] is None else st["pos"].long()
    # the rotation of pair (a, b) by an angle t as the complex product (a + ib) e^{it}
    turn = torch.complex(st["cos"].double(), st["sin"].double())[pos][:, None]

    def value(x, w):
        x = x.transpose(1, 2)
        y = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w
        a, b = _pair_halves(y, rot, inter)
        z = torch.complex(a.contiguous(), b.contiguous()) * turn
        z = torch.view_as_real(z)
        z = z.flatten(-2) if inter else z.transpose(-1, -2).flatten(-2)
        return torch.cat([z, y[..., rot:]], -1)

    out = {}
    for n in ("q", "k"):
        heads, grads, dw = [], [], 0
        w = st["w" + n].double()
        for h in range(st[n].shape[2]):         # a head at a time: the 64-bit intermediates are large
            x = st[n][:, :, h:h + 1].double()
            if not case["train"]:
                heads.append(value(x, w))
                continue
            x, wd = x.requires_grad_(), w.clone().requires_grad_()
            y = value(x, wd)
            dx, dwh = torch.autograd.grad(y, (x, wd), st["g" + n][:, h:h + 1].double())
            heads.append(y.detach())
            grads.append(dx)
            dw = dw + dwh
        out[n] = torch.cat(heads, 1)
        if case["train"]:
            out["d" + n] = torch.cat(grads, 2)
            out["dw" + n] = dw
    return out


def _exact_attn(case, st):
    G, Sq, Sk, d = case["Hq"] // case["Hkv"], case["Sq"], case["Sk"], case["d"]
    kv, start = _kv_lens(case), _q_starts(case)
    keys = {"out": st["q"], "lse": st["q"][..., 0]}
    if case["train"]:
        keys.update(dq=st["q"], dk=st["k"], dv=st["v"])
    out = {n: torch.zeros(x.shape, dtype=torch.float64, device="cuda") for n, x in keys.items()}
    j = torch.arange(Sk, device="cuda")
    for b in range(case["B"]):
        i = torch.arange(Sq, device="cuda") + start[b]
        seen = torch.zeros((Sq, Sk), dtype=torch.bool, device="cuda")
        seen[:, :kv[b]] = True
        if case["causal"]:
            order = i[:, None] >= j[None, :]
            if case["prefix"]:
                order[:, :_prefix_lens(case)[b]] = True
            seen &= order
        if case["doc"]:
            seen &= st["doc"][b][:, None] == st["doc"][b][None, :]
        for h in range(case["Hq"]):
            q = st["q"][b, h].double().requires_grad_(case["train"])
            k = st["k"][b, h // G].double().requires_grad_(case["train"])
            v = st["v"][b, h // G].double().requires_grad_(case["train"])
            s = q @ k.T / math.sqrt(d)
            if case["cap"]:
                s = case["cap"] * torch.tanh(s / case["cap"])
            if case["bias"]:
                s = s - st["slopes"][h].double() * (i[:, None] - j[None, :]).abs()
            s = s.masked_fill(~seen, -torch.inf)
            lse = torch.logsumexp(s, -1)
            p = torch.exp(s - torch.where(torch.isfinite(lse), lse, 0.0).detach()[:, None]) if not case["train"] \
                else torch.exp(s - torch.where(torch.isfinite(lse), lse, 0.0)[:, None])
            o = p @ v
            out["out"][b, h], out["lse"][b, h] = o.detach(), lse.detach()
            if case["train"]:
                dq, dk, dv = torch.autograd.grad(o, (q, k, v), st["g"][b, h].double())
                out["dq"][b, h] = dq
                out["dk"][b, h // G] += dk
                out["dv"][b, h // G] += dv
    return out


def exact(case, seed):
    st = prepare(case, seed)
    return _exact_norm(case, st) if case["op"] == "norm" else _exact_attn(case, st)
