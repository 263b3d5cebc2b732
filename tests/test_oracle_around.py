"""The fp64 forms of the norm with rotation and of attention over all keys: hand cases, and their
gradients against central differences."""
import numpy as np
import pytest

from oracle import around


def _differences(f, x, h=1e-5):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        y = x.copy()
        y[i] += h
        a = f(y)
        y[i] -= 2 * h
        g[i] = (a - f(y)) / (2 * h)
    return g


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("rot", [0, 4, 8])
def test_norm_rope_gradients_against_differences(interleaved, rot):
    rng = np.random.default_rng(rot)
    x, w, dy = rng.normal(size=(2, 3, 2, 8)), rng.normal(size=8), rng.normal(size=(2, 2, 3, 8))
    a = rng.normal(size=(5, rot // 2))
    cos, sin = (np.cos(a), np.sin(a)) if rot else (None, None)
    pos = rng.integers(0, 5, size=(2, 3))
    args = (cos, sin, pos, interleaved, 1e-3)
    dx, dw = around.norm_rope_grads(dy, x, w, *args)
    np.testing.assert_allclose(dx, _differences(lambda y: (around.norm_rope(y, w, *args) * dy).sum(), x), atol=1e-8)
    np.testing.assert_allclose(dw, _differences(lambda y: (around.norm_rope(x, y, *args) * dy).sum(), w), atol=1e-8)


def test_norm_rope_by_hand():
    # mean square 25/2 of (3, 4): r = sqrt(2)/5; a quarter turn takes (a, b) to (-b, a)
    x = np.array([3.0, 4.0]).reshape(1, 1, 1, 2)
    y = around.norm_rope(x, np.array([1.0, 2.0]), np.array([[0.0]]), np.array([[1.0]]), np.array([[0]]), True, 0.0)
    r = np.sqrt(2) / 5
    np.testing.assert_allclose(y.reshape(2), [-8 * r, 3 * r])


CASES = [dict(), dict(softcap=1.5), dict(causal=True), dict(causal=True, prefix_len=[3, 0]), dict(kv_len=[4, 0]),
         dict(slopes=[0.5, 0.25, -0.125, 1.0]), dict(q_start=[-2, 1], causal=True),
         dict(doc_q=[[0, 0, 1, -1], [2, 1, 1, 2]], doc_k=[[0, 1, 1, 0, -1], [1, 2, 3, 3, -1]], softcap=2.0)]


@pytest.mark.parametrize("case", CASES)
def test_dense_attention_gradients_against_differences(case):
    rng = np.random.default_rng(5)
    q, k, v = rng.normal(size=(2, 4, 4, 3)), rng.normal(size=(2, 2, 5, 3)), rng.normal(size=(2, 2, 5, 3))
    g = rng.normal(size=q.shape)
    r = around.dense_attention(q, k, v, dout=g, **case)
    for name, x, f in (("dq", q, lambda y: around.dense_attention(y, k, v, **case)),
                       ("dk", k, lambda y: around.dense_attention(q, y, v, **case)),
                       ("dv", v, lambda y: around.dense_attention(q, k, y, **case))):
        np.testing.assert_allclose(r[name], _differences(lambda y: (f(y)["out"] * g).sum(), x), atol=1e-7)


def test_dense_attention_by_hand():
    # two keys with scores 0 and log 3: weights 1/4 and 3/4
    q = np.ones((1, 1, 1, 1))
    k = np.array([0.0, np.log(3.0)]).reshape(1, 1, 2, 1)
    v = np.array([4.0, 8.0]).reshape(1, 1, 2, 1)
    r = around.dense_attention(q, k, v, scale=1.0)
    assert np.isclose(r["out"].item(), 7.0) and np.isclose(r["lse"].item(), np.log(4.0))
    r = around.dense_attention(q, k, v, scale=1.0, kv_len=[0])
    assert r["out"].item() == 0.0 and r["lse"].item() == -np.inf
    # a masked key may hold anything
    k[..., 1, :], v[..., 1, :] = np.nan, np.inf
    r = around.dense_attention(q, k, v, scale=1.0, kv_len=[1], dout=np.ones_like(q))
    assert r["out"].item() == 4.0 and r["dv"][0, 0, 1, 0] == 0.0 and r["dk"][0, 0, 1, 0] == 0.0


def test_visible_by_hand():
    see, p = around.visible(1, 2, 4, causal=True)
    assert see[0].tolist() == [[True, True, True, False], [True, True, True, True]] and p.tolist() == [[2, 3]]
    see, _ = around.visible(1, 2, 4, causal=True, q_start=[0], prefix_len=[2])
    assert see[0].tolist() == [[True, True, False, False], [True, True, False, False]]
    see, _ = around.visible(1, 2, 3, doc_q=[[1, -1]], doc_k=[[1, -1, 2]])
    assert see[0].tolist() == [[True, False, False], [False, False, False]]
