"""Pins of the routed oracle (CPU): brute force over all selections, exhaustive
ties, the existing router oracle, and central differences."""
import itertools
import math

import numpy as np
import pytest

import oracle


def _brute(l, bias, k, score, G, Gk, gtop, renorm, scale):
    """One row by maximising over all choices of groups and experts."""
    E = len(l)
    on = [i for i in range(E) if l[i] > -math.inf]
    if score == "sigmoid":
        s = {i: 1.0 / (1.0 + math.exp(-l[i])) for i in on}
    else:
        z = sum(math.exp(l[i]) for i in on)
        s = {i: math.exp(l[i]) / z for i in on}
    c = {i: s[i] + (bias[i] if bias is not None else 0.0) for i in on}
    gs = E // G

    def group_score(g):
        return sum(sorted((c[i] for i in on if i // gs == g), reverse=True)[:gtop])

    live = [g for g in range(G) if any(i // gs == g for i in on)]
    n = min(Gk, len(live))
    kept = max(itertools.combinations(live, n), key=lambda gg: sum(group_score(g) for g in gg)) if n else ()
    cand = [i for i in on if i // gs in kept]
    m = min(k, len(cand))
    best = max(itertools.permutations(cand, m), key=lambda ii: sum(c[i] * 10.0 ** -j for j, i in enumerate(ii))
               + 1e6 * sum(c[i] for i in ii)) if m else ()
    best = sorted(best, key=lambda i: -c[i])
    S = sum(s[i] for i in best) if renorm else 1.0
    return list(best) + [-1] * (k - m), [scale * s[i] / S for i in best] + [0.0] * (k - m)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("G,Gk,gtop", [(1, 1, 1), (3, 2, 1), (3, 2, 2), (3, 1, 2)])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("with_bias", [True, False])
def test_route_equals_the_maximum_over_all_selections(score, G, Gk, gtop, renorm, with_bias):
    rng = np.random.default_rng(3)
    T, E, k = 40, 9, 2
    l = rng.standard_normal((T, E))
    l[rng.random((T, E)) < 0.3] = -np.inf
    bias = 0.3 * rng.standard_normal(E) if with_bias else None
    ids, w, _ = oracle.route_logits(l, bias, k, score, G, Gk, gtop, renorm, 1.5)
    for t in range(T):
        want_ids, want_w = _brute(l[t], bias, k, score, G, Gk, gtop, renorm, 1.5)
        assert list(ids[t]) == want_ids
        assert np.allclose(w[t], want_w, rtol=1e-12, atol=0)


def test_route_ties_go_to_the_lower_index_everywhere():
    for vals in itertools.product([0.0, 1.0, -1.0], repeat=4):
        l = np.array([vals])
        for score in ("sigmoid", "softmax"):
            ids, _, _ = oracle.route_logits(l, None, 2, score)
            assert list(ids[0]) == sorted(range(4), key=lambda i: (-vals[i], i))[:2]
            ids, _, _ = oracle.route_logits(l, None, 1, score, 2, 1, 2)
            g = 0 if sum(map(lambda v: oracle.route_scores(l[0], score)[v], (0, 1))) >= \
                sum(map(lambda v: oracle.route_scores(l[0], score)[v], (2, 3))) else 1
            assert ids[0, 0] == max((2 * g, 2 * g + 1), key=lambda i: (vals[i], -i))


def test_route_without_groups_and_bias_is_the_router_of_the_layer():
    rng = np.random.default_rng(4)
    l = rng.standard_normal((64, 12))
    for gating, score, renorm in ((oracle.SOFTMAX_ALL_RENORM, "softmax", True),
                                  (oracle.SIGMOID_TOPK_RENORM, "sigmoid", True),
                                  (oracle.SOFTMAX_ALL_NO_RENORM, "softmax", False)):
        ids, w, _ = oracle.route_logits(l, None, 3, score, renormalise=renorm)
        want = oracle.topk_select(l, 3)
        assert np.array_equal(ids, want)
        assert np.allclose(w, oracle.gate_weights(l, None, want, gating), rtol=1e-12)


def test_masks_and_empty_rows():
    low = float(np.finfo(np.float32).min)
    l = np.array([[np.nan, -np.inf, low, 2.0, np.inf], [low] * 5, [-np.inf] * 5])
    ids, w, _ = oracle.route_logits(l, None, 3, "sigmoid")
    assert ids.tolist() == [[4, 3, -1], [-1] * 3, [-1] * 3]
    assert np.allclose(w[0], np.array([1.0, 1 / (1 + math.exp(-2.0)), 0.0]) / (1.0 + 1 / (1 + math.exp(-2.0))))
    assert not w[1:].any()
    ids, w, _ = oracle.route_logits(np.array([[-900.0, -901.0, -2000.0]]), None, 2, "sigmoid")
    assert np.allclose(w[0], np.array([1.0, math.exp(-1)]) / (1 + math.exp(-1)))
    _, w, _ = oracle.route_logits(np.array([[1e30, 1e30, 0.0]]), None, 2, "softmax", renormalise=False)
    assert w.tolist() == [[0.5, 0.5]] or np.allclose(w, 0.5, rtol=1e-15)
    ids, _, _ = oracle.route_logits(np.zeros((1, 3)), np.array([-np.inf, np.nan, -50.0]), 2, "softmax")
    assert ids.tolist() == [[2, -1]]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("balance,z,weights", [(0.0, 0.0, True), (0.7, 0.0, True), (0.0, 0.3, True),
                                               (0.7, 0.3, True), (0.7, 0.3, False)])
def test_route_backward_against_central_differences(score, renorm, balance, z, weights):
    """Central differences with step h have an error of h^2/6 times the third
    derivative (of order 1 here: scores of logits of order 1) plus the
    objective's rounding, 2^-53 |objective| / h < 1e-15 * 10 / 1e-5: below
    1e-8 in all."""
    rng = np.random.default_rng(5)
    T, E, k = 5, 7, 3
    l = rng.standard_normal((T, E))
    l[0, 2] = -np.inf
    l[3] = -np.inf
    ids, _, _ = oracle.route_logits(l, 0.1 * rng.standard_normal(E), k, score)
    ids[4, 1] = -1
    g = rng.standard_normal((T, k)) if weights else None
    counts = np.bincount(ids[ids >= 0], minlength=E)
    args = (ids, g, score, renorm, 2.5, counts, balance, z)
    got = oracle.route_backward(l, *args)
    for t in range(T):
        for e in range(E):
            if not l[t, e] > -np.inf:
                assert got[t, e] == 0.0
                continue
            lo, hi = l.copy(), l.copy()
            lo[t, e] -= 1e-5
            hi[t, e] += 1e-5
            want = (oracle.route_objective(hi, *args) - oracle.route_objective(lo, *args)) / 2e-5
            assert abs(got[t, e] - want) < 1e-8


def test_objective_penalties_are_the_layers():
    rng = np.random.default_rng(6)
    l = rng.standard_normal((20, 6))
    counts = np.array([3, 0, 9, 1, 5, 2])
    ids = np.full((20, 1), -1)
    assert math.isclose(oracle.route_objective(l, ids, None, "sigmoid", True, 1.0, counts, balance=1.0),
                        oracle.balance_loss(l, counts), rel_tol=1e-12)
    assert math.isclose(oracle.route_objective(l, ids, None, "sigmoid", True, 1.0, z=1.0), oracle.router_z_loss(l),
                        rel_tol=1e-12)


def test_combine_backward_against_differences_of_combine():
    """combine is linear in either argument, so a difference of step 1 is exact
    up to rounding (values of order 1, 2^-50)."""
    rng = np.random.default_rng(7)
    T, k, d = 4, 2, 3
    row_of = np.array([2, 5, 0, -1, 1, 3, -1, 4])
    yp, w, gy = rng.standard_normal((8, d)), rng.random((T, k)), rng.standard_normal((T, d))
    rows, gw = oracle.combine_backward(gy, yp, row_of, w, k)

    def f(yp, w):
        return float(np.sum(gy * oracle.combine(yp, row_of, w)))
    for r in range(8):
        for j in range(d):
            q = yp.copy()
            q[r, j] += 1.0
            want = f(q, w) - f(yp, w)
            assert (r in (6, 7) and np.isnan(rows[r, j])) or abs(rows[r, j] - want) < 1e-12
    for t in range(T):
        for s in range(k):
            q = w.copy()
            q[t, s] += 1.0
            assert abs(gw[t, s] - (f(yp, q) - f(yp, w))) < 1e-12


def test_adapters_equal_experts_with_the_update_merged_into_the_weights():
    """(W + s B A) x = W x + s B (A x), per adapter and expert."""
    rng = np.random.default_rng(8)
    N, E, r, d, f, rows = 3, 2, 4, 6, 5, 12
    w, wd = rng.standard_normal((E, 2 * f, d)), rng.standard_normal((E, d, f))
    a, b = rng.standard_normal((N, E, r, d)), rng.standard_normal((N, E, 2 * f, r))
    ad, bd = rng.standard_normal((N, E, r, f)), rng.standard_normal((N, E, d, r))
    s = rng.random(N)
    x = rng.standard_normal((rows, d))
    adapter, expert = rng.integers(-1, N + 1, rows), rng.integers(0, E, rows)
    pre = np.stack([w[expert[i]] @ x[i] for i in range(rows)])
    h = oracle.adapter_gate_up(x, adapter, expert, a, b, s, pre, oracle.ACT_SWIGLU)
    base = np.stack([wd[expert[i]] @ h[i] for i in range(rows)])
    y = oracle.adapter_down(h, adapter, expert, ad, bd, s, base)
    for i in range(rows):
        n, e = adapter[i], expert[i]
        m = w[e] + (s[n] * b[n, e] @ a[n, e] if 0 <= n < N else 0.0)
        md = wd[e] + (s[n] * bd[n, e] @ ad[n, e] if 0 <= n < N else 0.0)
        want = oracle.swiglu_expert(x[i:i + 1], m[:f], m[f:], md)
        assert np.allclose(y[i], want[0], rtol=1e-10, atol=1e-12)
    g = oracle.adapter_gate_up(x, adapter, expert, a, b, s, pre, oracle.ACT_GELU)
    assert np.allclose(g, oracle.gelu(pre + oracle.adapter_delta(x, adapter, expert, a, b, s)))
