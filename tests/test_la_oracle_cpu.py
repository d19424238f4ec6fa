"""The float64 oracle of linear attention with a decay for each head: its gradients against central
differences, and a state that is cleared."""
import numpy as np

from oracle import la


def inputs(T, dk, dv, seed):
    r = np.random.default_rng(seed)
    return [r.standard_normal((T, dk)), r.standard_normal((T, dk)), r.standard_normal((T, dv)), -r.random(T),
            r.standard_normal((T, dv)), r.standard_normal((dk, dv)), r.standard_normal((dk, dv))]


def loss(q, k, v, g, dO, dS, S0):
    o, M = la.la_recurrent(q, k, v, g, S0)
    return np.sum(o * dO) + np.sum(M[-1] * dS)


def test_gradients_against_differences():
    x = inputs(6, 3, 4, 1)
    d = la.la_backward(*x)
    h = 1e-5
    for at, name in ((0, "dq"), (1, "dk"), (2, "dv"), (3, "dg"), (6, "dS0")):
        for i in np.ndindex(x[at].shape):
            up, down = [y.copy() for y in x], [y.copy() for y in x]
            up[at][i] += h
            down[at][i] -= h
            assert abs((loss(*up) - loss(*down)) / (2 * h) - d[name][i]) < 1e-7, (name, i)


def test_a_cleared_state_forgets():
    q, k, v, g, dO, dS, S0 = inputs(7, 3, 4, 2)
    g[4] = -np.inf
    o, M = la.la_recurrent(q, k, v, g, S0)
    o2, M2 = la.la_recurrent(q[4:], k[4:], v[4:], g[4:])
    assert np.array_equal(o[4:], o2) and np.array_equal(M[-1], M2[-1])
    d = la.la_backward(q, k, v, g, dO, dS, S0)
    assert d["dg"][4] == 0 and np.all(np.isfinite(d["dg"]))
