"""Caps of any size over scores of any size: a cap far above the scores leaves them as they are, one far
below makes them signs, and the values' magnitude is the caller's. The bounds are those of dense_cases
but for the cap: tanh is off by 2^-20 of its own value at most (a polynomial whose leading
coefficient is 1 - 3.6e-7, or 1 - 2 / (1 + e^2y) above y = 1, and a few half steps of fp32), so a score by
2^-20 of itself, whatever the cap."""
import numpy as np
import pytest
import torch

import block_sparse_top_fvattn_b200 as fv
from dense_cases import F, HALF, draw, f64, reference, run

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fv.load()


def forward_within(x, cfg, dtype):
    got = run(x, cfg, grads=False)
    r = reference(x, cfg, grads=False)
    d, Sk = r["q"].shape[-1], r["k"].shape[2]
    qk = np.einsum("bhid,bhjd->bhij", np.abs(r["q"]), np.abs(r["k"])) * r["scale"]
    qk = np.minimum(qk, 1e30)
    s = np.abs(np.einsum("bhid,bhjd->bhij", r["q"], r["k"]) * r["scale"])
    s = cfg.softcap * np.tanh(s / cfg.softcap)                # the capped score's magnitude
    # an error of the product reaches the score times the cap's derivative
    fin = np.abs(r["lse"])[..., None]
    e = (2 * d + 8) * F * qk * r["cap"] + (2.0 ** -20 + 8 * F) * s + 8 * F * fin + 2.0 ** -21
    rel = 2 * np.where(r["p"] > 0, e, 0.0).max(axis=-1, keepdims=True)
    u = HALF[dtype]
    acc = (Sk + 8) * 2 * F
    A = np.einsum("bhij,bhjd->bhid", r["p"], np.abs(r["v"]))
    tol = (rel + acc + (u if dtype == BF16 else 0.0)) * A + u * np.abs(r["out"]) + 1e-30
    far = np.abs(f64(got["out"]) - r["out"]) / tol
    assert far.max() <= 1.0, f"out: {far.max():.2f} times its bound"
    far = np.abs(f64(got["lse"]) - r["lse"]) / ((rel + acc)[..., 0] + 8 * F * fin[..., 0])
    assert far.max() <= 1.0, f"lse: {far.max():.2f} times its bound"


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cap", [1e-20, 1e-3, 1e3, 1e4, 1e6, 1e20])
@pytest.mark.parametrize("shape", [(2, 4, 2, 1, 500, 128), (1, 4, 1, 3, 300, 64), (1, 4, 2, 100, 200, 64)])
def test_any_cap(dtype, cap, shape):
    # up to 16 rows of a shared key head, and more
    forward_within(draw(*shape, dtype, seed=1, spread=2.0), fv.AttnConfig(softcap=cap), dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Sq", [1, 4, 40])
def test_small_scores_beside_large_ones(dtype, Sq):
    # one head's scores reach 7 times the cap of 1e6, the others' are of the order of one
    x = draw(1, 4, 1, Sq, 300, 64, dtype, seed=2, spread=2.0)
    x["q"][:, 1] = x["q"][:, 1] * 1e6
    x["k"][:, :, 7] *= 4
    forward_within(x, fv.AttnConfig(softcap=1e6), dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gradients_of_small_scores_beside_large_ones(dtype):
    # per head: what the large head does must not change the others' gradients beyond their roundings
    x = draw(1, 4, 4, 130, 200, 64, dtype, seed=3, spread=2.0)
    x["q"][:, :, 5] *= 1e7                      # one row of every head
    cfg = fv.AttnConfig(softcap=1e6)
    got, r = run(x, cfg), reference(x, cfg)
    u = HALF[dtype]
    keep = np.arange(130) != 5
    # P and dS rounded to the inputs' type, dq rounded: their magnitudes bound the error
    ds, p = np.abs(r["ds"]), r["p"]
    rel = 2.0 ** -12                            # of the weights: scores below 40 off by (2 d + 16) F + 2^-20 of themselves
    e_ds = ds * (u + 2 * rel) + p * r["scale"] * (rel + 2.0 ** -13) * \
        np.einsum("bhid,bhjd->bhij", np.abs(r["g"]), np.abs(r["v"]))
    tol = np.einsum("bhij,bhjd->bhid", e_ds, np.abs(r["k"])) + u * np.abs(r["dq"]) + 1e-30
    far = (np.abs(f64(got["dq"]) - r["dq"]) / tol)[:, :, keep]
    assert far.max() <= 1.0, f"dq: {far.max():.2f} times its bound"


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cap", [5.0, 30.0, 50.0, 51.0])
@pytest.mark.parametrize("size", [2.0 ** 100, 2.0 ** -100])
@pytest.mark.parametrize("Sq", [130, 1])
def test_values_of_any_size(dtype, cap, size, Sq):
    # every score at the cap or at its negative: out is the mean of the values, as large or small as they are
    Sk, d = 300, 64
    x = draw(1, 2, 1, Sq, Sk, d, dtype)
    sign = torch.ones(Sq, device="cuda")
    sign[::2] = -1
    x["q"] = (sign[:, None] * torch.ones(1, 2, Sq, d, device="cuda")).to(dtype)
    x["k"] = torch.ones(1, 1, Sk, d, device="cuda").to(dtype)
    x["v"] = x["v"] * size
    got = run(x, fv.AttnConfig(softcap=cap), grads=False, scale=25.0 * cap / d)
    v = f64(x["v"])
    u = HALF[dtype]
    mean, mag = v.mean(axis=2, keepdims=True), np.abs(v).mean(axis=2, keepdims=True)
    # the weight's rounding and the sum of Sk terms on mean |v|, the rounding of out
    tol = (u + (Sk + 8) * 2 * F) * mag + u * np.abs(mean)
    far = np.abs(f64(got["out"]) - mean) / tol
    assert far.max() <= 1.0, f"{far.max():.2f} times its bound"
