"""The norm's gradients where a CTA takes several tiles of tokens one after the other: the carried sums of
the weights' gradients, a ragged last range, the number of partial rows. fp64 values on the device."""
import pytest
import torch

import block_sparse_top_fvattn_b200 as fv

pytestmark = pytest.mark.gpu

F = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fv.load()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,S,Hq,Hk,d", [(1, 160001, 2, 2, 128), (3, 100003, 1, 1, 64), (1, 80007, 3, 33, 128)])
def test_gradients_of_many_tokens(dtype, B, S, Hq, Hk, d):
    # tiles of 16 (d = 128) or 32 tokens: 10001 and 9376 tiles of two groups of heads, 5001 of four (a CTA then
    # takes 4, 3 and 4 tiles, the last of each a ragged range)
    g = torch.Generator(device="cuda").manual_seed(0)
    n = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)      # noqa: E731
    xs = {"q": n(B, S, Hq, d), "k": n(B, S, Hk, d)}
    gs = {"q": n(B, Hq, S, d), "k": n(B, Hk, S, d)}
    ws = {"q": 1 + 0.2 * torch.randn(d, generator=g, device="cuda"), "k": 1 + 0.2 * torch.randn(d, generator=g, device="cuda")}
    ang = torch.arange(S, device="cuda", dtype=torch.float64)[:, None] * \
        10000.0 ** (-torch.arange(0, d, 2, device="cuda", dtype=torch.float64) / d)
    cos, sin = ang.cos().float(), ang.sin().float()
    dq, dk, dwq, dwk = fv.qk_norm_rope_bwd(gs["q"], gs["k"], xs["q"], xs["k"], ws["q"], ws["k"], cos, sin)
    got = {"q": (dq, dwq), "k": (dk, dwk)}
    u = 2.0 ** -8 if dtype == torch.bfloat16 else F
    c, s = cos.double()[None], sin.double()[None]
    for t in ("q", "k"):
        dx, dw = got[t]
        w = ws[t].double()
        total, size, least = torch.zeros(d, dtype=torch.float64, device="cuda"), 0.0, None
        for h in range(xs[t].shape[2]):
            x = xs[t][:, :, h].double()
            dy = gs[t][:, h].double()
            a, b = dy[..., 0::2], dy[..., 1::2]
            gr = torch.stack([a * c + b * s, b * c - a * s], -1).flatten(-2)
            # what the rotation's two products and their sum may be off by, in units of F
            turned = torch.stack([(a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()], -1).flatten(-2)
            r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6)
            term = gr * r * x
            total += term.sum((0, 1))
            size = size + (turned * r * x.abs()).sum((0, 1))
            row = term[-1, -1].abs()                       # the last token's, of the ragged range
            least = row if least is None else torch.maximum(least, row)
            gw = gr * w
            want = r * gw - x * r ** 3 * (gw * x).mean(-1, keepdim=True)
            mag = r * turned * w.abs() + x.abs() * r ** 3 * (turned * w.abs() * x.abs()).mean(-1, keepdim=True)
            far = (dx[:, :, h].double() - want).abs() / (2 * (d + 32) * F * mag + u * want.abs() + 1e-30)
            assert far.max().item() <= 1.0, f"d{t}: {far.max().item():.2f} times its bound"
        # A thread adds the terms of its token in each of at most 4 tiles and 16 heads, a CTA those of at most 32
        # tokens, in fp32; the rest in fp64. A term: the rotation (3), r (d / 8 + 4 shuffles + 4, halved by the
        # root) and three products.
        bound = (64 + 32 + 3 + d // 16 + 4 + 3) * F * size + F * total.abs()
        far = (dw.double() - total).abs() / bound
        assert far.max().item() <= 1.0, f"dw{t}: {far.max().item():.2f} times its bound"
        # a sum that misses one row is outside the bound in some column
        assert (least > bound).any() or xs[t].shape[2] > 16
