"""The fp64 oracle of the attention layer and the update against central differences of its own forward, and
hand-computed values.  CPU only."""
import numpy as np
import pytest

from oracle import attn_oracle as ao

H = 1e-5  # truncation H^2 times a third derivative (|x| here is O(1)) and rounding 1e-16 / H: both below 1e-8


def _diff(f, x, at):
    y = x.copy()
    y[at] += H
    up = f(y)
    y[at] -= 2 * H
    return (up - f(y)) / (2 * H)


@pytest.mark.parametrize("lq,lk,Hq,Hkv,causal", [([3, 2], [3, 2], 2, 1, True), ([4], [6], 4, 2, True),
                                                 ([5], [2], 2, 2, True), ([3, 0], [4, 3], 3, 1, False)])
def test_attention_gradients_against_differences(lq, lk, Hq, Hkv, causal):
    r = np.random.default_rng(0)
    D = 4
    q, k, v, w = (r.normal(size=(n, h, D)) for n, h in ((sum(lq), Hq), (sum(lk), Hkv), (sum(lk), Hkv), (sum(lq), Hq)))
    seqs = ao.sequences(np.concatenate([[0], np.cumsum(lq)]), np.concatenate([[0], np.cumsum(lk)]))
    f = lambda a, b, c: float((ao.attention(a, b, c, seqs, causal, 0.7)["out"] * w).sum())  # noqa: E731
    g = ao.attention(q, k, v, seqs, causal, 0.7, dout=w)
    for name, i in (("dq", 0), ("dk", 1), ("dv", 2)):
        args = [q, k, v]
        for at in np.ndindex(args[i].shape):
            d = _diff(lambda x: f(*[x if j == i else args[j] for j in range(3)]), args[i], at)
            assert abs(d - g[name][at]) < 1e-7, (name, at)


def test_attention_by_hand():
    """Two keys of equal score share a query's weight; a query before both sees nothing."""
    k = np.zeros((2, 1, 2))
    v = np.array([[[1.0, 2.0]], [[3.0, 6.0]]])
    r = ao.attention(np.ones((3, 1, 2)), k, v, [(0, 3, 0, 2)], True, 1.0)
    assert np.allclose(r["out"][:, 0], [[0, 0], [1, 2], [2, 4]])
    assert r["lse"][0, 0] == -np.inf and np.allclose(r["lse"][0, 1:], [0, np.log(2)])


@pytest.mark.parametrize("norm,R", [(True, 8), (True, 4), (False, 8)])
def test_norm_rotation_gradients_against_differences(norm, R):
    r = np.random.default_rng(1)
    x, w = r.normal(size=(3, 2, 8)), r.normal(size=(3, 2, 8))
    g = r.normal(size=8) if norm else None
    pos, inv = np.array([0, 5, 1000]), 10.0 ** -np.arange(R // 2)
    f = lambda a, b: float((ao.qk_norm_rope(a, b, pos, inv, 1e-3) * w).sum())  # noqa: E731
    dx, dg = ao.qk_norm_rope_bwd(w, x, g, pos, inv, 1e-3)
    for at in np.ndindex(x.shape):
        assert abs(_diff(lambda y: f(y, g), x, at) - dx[at]) < 1e-7
    for at in np.ndindex(g.shape) if norm else ():
        assert abs(_diff(lambda y: f(x, y), g, at) - dg[at]) < 1e-7


def test_adamw_by_hand():
    """First step from zero states: m / (1 - b1) = g and sqrt(v / (1 - b2)) = |g|, so p moves by lr sign(g)."""
    p, m, v, _, _ = ao.adamw(np.array([1.0, 2.0]), np.array([3.0, -0.5]), np.zeros(2), np.zeros(2), 1, 0.1, 0.9, 0.95, 0.0,
                             0.5)
    assert np.allclose(p, [0.95 - 0.1, 1.9 + 0.1]) and np.allclose(m, [0.3, -0.05]) and np.allclose(v, [0.45, 0.0125])
