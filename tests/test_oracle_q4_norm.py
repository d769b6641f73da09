"""Pins of the oracles of the 4-bit linears and the block norms: brute force,
closed cases, and differences for the gradients."""
import numpy as np
import pytest

from oracle import nq_norm as N
from oracle import nq_q4 as Q


@pytest.mark.parametrize("m,n,G,zeros", [(3, 5, 32, False), (4, 70, 32, True), (2, 200, 64, True), (5, 128, 128, False)])
def test_q4_linear_is_the_sum_over_columns(m, n, G, zeros):
    rng = np.random.default_rng([1, m, n, G])
    q, ng = rng.integers(0, 16, (m, n)), -(-n // G)
    s, z = rng.standard_normal((m, ng)), rng.integers(0, 16, (m, ng)) if zeros else None
    x = rng.standard_normal((3, n))
    got = Q.linear(x, q, s, z, G)
    for b in range(3):
        for i in range(m):
            want = sum(s[i, j // G] * (int(q[i, j]) - (int(z[i, j // G]) if zeros else 8)) * x[b, j] for j in range(n))
            assert abs(got[b, i] - want) <= 1e-12 * Q.magnitude(x, q, s, z, G)[b, i]


def test_q4_code_equal_to_its_zero_point_is_zero():
    assert not Q.weight(np.full((2, 40), 8), np.ones((2, 2)), None, 32).any()
    assert not Q.weight(np.full((2, 40), 3), np.ones((2, 2)), np.full((2, 2), 3), 32).any()


def test_norm_of_a_row_of_equal_values():
    h, x = N.forward(np.full((1, 6), 2.0), np.full((1, 6), -5.0), None, np.full(6, 3.0), None, 1.0, 0.5, 0.0)
    assert np.allclose(h, 1.5) and np.allclose(x, 3.0)  # post(-5) = -1, 2 - 0.5 = 1.5, pre = 1, times 3


CASES = [(post, pre, gate) for post in (True, False) for pre in (True, False) for gate in (None, "channel", "rows")]


@pytest.mark.parametrize("post,pre,gate", CASES)
def test_norm_gradients_against_differences(post, pre, gate):
    """d/dtheta of L = sum(x dx) + sum(h' dh) by central differences of step e in
    fp64: off by O(e^2) + 1e-16 / e, about 1e-9 relative at e = 1e-5."""
    rng = np.random.default_rng([2, post, pre, gate == "rows"])
    rows, d, a, b, eps = 3, 5, 0.9, 0.7, 1e-2
    p = {"h": rng.standard_normal((rows, d)), "y": rng.standard_normal((rows, d)), "wp": 1 + rng.random(d),
         "wq": 1 + rng.random(d)}
    if gate:
        p["gate"] = rng.standard_normal(d if gate == "channel" else (rows, d))
    dx, dh = rng.standard_normal((rows, d)), rng.standard_normal((rows, d))

    def loss(p):
        ho, x = N.forward(p["h"], p["y"], p["wp"], p["wq"], p.get("gate"), a, b, eps, post, pre)
        return np.sum(ho * dh) + (np.sum(x * dx) if pre else 0.0)

    ho, _ = N.forward(p["h"], p["y"], p["wp"], p["wq"], p.get("gate"), a, b, eps, post, pre)
    out = N.backward(dx, dh, ho, p["y"], p["wp"], p["wq"], p.get("gate"), a, b, N.rstd(p["y"], eps), N.rstd(ho, eps),
                     post, pre)
    want = {"h": out["h"], "y": out["y"]}
    if post:
        want["wp"] = out["w_post"]
    if pre:
        want["wq"] = out["w_pre"]
    if gate:
        want["gate"] = out["gate"].sum(0) if gate == "channel" else out["gate"]
    for k, g in want.items():
        for at in np.ndindex(p[k].shape):
            ends = []
            for step in (1e-5, -1e-5):
                q = {n: v.copy() for n, v in p.items()}
                q[k][at] += step
                ends.append(loss(q))
            assert abs((ends[0] - ends[1]) / 2e-5 - g[at]) <= 1e-7 * (1 + abs(g[at])), (k, at)


def test_norm_gradient_without_a_block():
    """y None: h' = h, and the gradient of h is that of h' through the pre norm alone."""
    rng = np.random.default_rng(3)
    h, dx, w = rng.standard_normal((2, 4)), rng.standard_normal((2, 4)), 1 + rng.random(4)
    out = N.backward(dx, None, h, None, None, w, None, 9.0, 9.0, None, N.rstd(h, 1e-2))
    for at in np.ndindex(h.shape):
        ends = []
        for step in (1e-5, -1e-5):
            k = h.copy()
            k[at] += step
            ends.append(np.sum(N.forward(k, None, None, w, None, 9.0, 9.0, 1e-2)[1] * dx))
        assert abs((ends[0] - ends[1]) / 2e-5 - out["h"][at]) <= 1e-7 * (1 + abs(out["h"][at]))
