"""Plain CPU statement of routing from logits, of its gradient, of the
combine's gradient and of low-rank adapters beside the experts' projections.

TEST INFRASTRUCTURE ONLY, like ``moe_oracle``.  Everything is float64, written
row by row from the formulas; pinned by ``tests/test_routed_pins.py`` against
brute force, exhaustive tiny cases and central differences.

Definitions (per token): an expert is available when its logit is above the
lowest finite value of the stored type and its bias is neither -inf nor NaN;
scores are sigmoids, or the softmax over the available *logits*; the choice is
score + bias; groups are equal blocks of neighbouring experts, scored by their
largest choice or the sum of their two largest; ties go to the lower index.
"""
from __future__ import annotations

import math

import numpy as np

from .moe_oracle import ACT_SWIGLU, gelu, silu

__all__ = ["usable_logits", "route_scores", "route_logits", "route_objective", "route_backward",
           "combine_backward", "adapter_delta", "adapter_gate_up", "adapter_down"]

LOWEST = {"f32": -float(np.finfo(np.float32).max), "bf16": -3.3895313892515355e38}
F32_MAX = float(np.finfo(np.float32).max)


def usable_logits(logits, dtype: str) -> np.ndarray:
    """The logits with -inf in masked places (-inf, NaN, the type's lowest
    value) and +inf as the largest finite float32."""
    l = np.array(logits, dtype=np.float64, copy=True)
    with np.errstate(invalid="ignore"):
        l[~(l > LOWEST[dtype])] = -np.inf
    return np.minimum(l, F32_MAX)


def route_scores(l: np.ndarray, score: str) -> np.ndarray:
    """Scores of one row of usable logits (0 in masked places)."""
    s = np.zeros(len(l))
    on = l > -np.inf
    if not on.any():
        return s
    if score == "sigmoid":
        for i in np.nonzero(on)[0]:
            s[i] = 1.0 / (1.0 + math.exp(-l[i])) if l[i] > -700.0 else 0.0
    else:
        m = l[on].max()
        e = np.exp(l[on] - m)
        s[on] = e / e.sum()
    return s


def _log_score(l_i: float, row: np.ndarray, score: str) -> float:
    if score == "sigmoid":
        return -math.log1p(math.exp(-l_i)) if l_i > 0 else l_i - math.log1p(math.exp(l_i))
    on = row[row > -np.inf]
    return (l_i - on.max()) - math.log(np.exp(on - on.max()).sum())


def route_logits(logits, bias, k: int, score: str, n_groups: int = 1, topk_groups: int = 1, group_top: int = 1,
                 renormalise: bool = True, scale: float = 1.0, dtype: str = "f32"):
    """-> (ids [T, k], w [T, k], gap [T]): the picks, their weights and the
    smallest difference between choices (or group scores) that decided
    something, so a test can tell rows that hang on a rounding."""
    l = usable_logits(logits, dtype)
    T, E = l.shape
    gs = E // n_groups
    ids = np.full((T, k), -1, dtype=np.int64)
    w = np.zeros((T, k))
    gap = np.full(T, np.inf)
    for t in range(T):
        s = route_scores(l[t], score)
        c = s + (np.asarray(bias, dtype=np.float64) if bias is not None else 0.0)
        c[~(c > -np.inf)] = -np.inf
        c[~(l[t] > -np.inf)] = -np.inf
        if n_groups > 1:
            sums = []
            for g in range(n_groups):
                best = sorted((v for v in c[g * gs:(g + 1) * gs] if v > -np.inf), reverse=True)[:group_top]
                sums.append(sum(best) if best else -np.inf)
            order = sorted(range(n_groups), key=lambda g: (-sums[g], g))
            if topk_groups < n_groups and sums[order[topk_groups]] > -np.inf:
                gap[t] = sums[order[topk_groups - 1]] - sums[order[topk_groups]]
            for g in order[topk_groups:]:
                c[g * gs:(g + 1) * gs] = -np.inf
        # equal scores of different logits (saturation) still rank by the logit
        order = [i for i in sorted(range(E), key=lambda i: (-c[i], -l[t, i] if bias is None else 0.0, i))
                 if c[i] > -np.inf]
        for a, b in zip(order[:k], order[1:k + 1]):
            gap[t] = min(gap[t], c[a] - c[b])
        lw = [_log_score(l[t, i], l[t], score) for i in order[:k]]
        if renormalise and lw:
            m = max(lw)
            lz = m + math.log(sum(math.exp(v - m) for v in lw))
            lw = [v - lz for v in lw]
        for j, i in enumerate(order[:k]):
            ids[t, j] = i
            w[t, j] = scale * math.exp(lw[j])
    return ids, w, gap


def route_objective(logits, ids, grad_w, score: str, renormalise: bool, scale: float, counts=None,
                    balance: float = 0.0, z: float = 0.0, dtype: str = "f32") -> float:
    """sum grad_w * w(ids) + balance * E sum_e f_e mean_t p + z * mean_t lse^2,
    the scalar whose gradient ``route_backward`` is (ids fixed)."""
    l = usable_logits(logits, dtype)
    T, E = l.shape
    total = 0.0
    f = None
    if balance:
        n = float(np.sum(counts))
        f = np.asarray(counts, dtype=np.float64) / n if n > 0 else np.zeros(E)
    for t in range(T):
        s = route_scores(l[t], score)
        got = [(j, i) for j, i in enumerate(ids[t]) if 0 <= i < E and l[t, i] > -np.inf]
        if got and grad_w is not None:
            S = sum(s[i] for _, i in got) if renormalise else 1.0
            total += sum(grad_w[t, j] * scale * s[i] / S for j, i in got)
        on = l[t] > -np.inf
        if not on.any():
            continue
        p = route_scores(l[t], "softmax")
        if balance:
            total += balance * E * float(f @ p) / T
        if z:
            m = l[t][on].max()
            total += z * (m + math.log(np.exp(l[t][on] - m).sum())) ** 2 / T
    return total


def route_backward(logits, ids, grad_w, score: str, renormalise: bool, scale: float, counts=None,
                   balance: float = 0.0, z: float = 0.0, dtype: str = "f32") -> np.ndarray:
    """d route_objective / d logits from the Jacobians, row by row."""
    l = usable_logits(logits, dtype)
    T, E = l.shape
    out = np.zeros((T, E))
    f = np.zeros(E)
    if balance and np.sum(counts) > 0:
        f = np.asarray(counts, dtype=np.float64) / float(np.sum(counts))
    for t in range(T):
        on = l[t] > -np.inf
        if not on.any():
            continue
        p = route_scores(l[t], "softmax")
        s = p if score == "softmax" else route_scores(l[t], score)
        ds = np.zeros(E)  # d objective / d scores
        got = [(j, i) for j, i in enumerate(ids[t]) if 0 <= i < E and on[i]]
        if grad_w is not None and got:
            S = sum(s[i] for _, i in got)
            dot = sum(grad_w[t, j] * s[i] for j, i in got)
            for j, i in got:
                if not renormalise:
                    ds[i] += scale * grad_w[t, j]
                elif S > 0:
                    ds[i] += scale * (grad_w[t, j] / S - dot / S ** 2)
        if score == "sigmoid":
            out[t] = ds * s * (1.0 - s)
        else:
            out[t] = p * (ds - p @ ds)
        if balance:
            v = balance * E / T * f
            out[t] += p * (v - p @ v)
        if z:
            m = l[t][on].max()
            out[t] += 2.0 * z / T * (m + math.log(np.exp(l[t][on] - m).sum())) * p
        out[t][~on] = 0.0
    return out


def combine_backward(grad_y, y_perm, row_of, w, k: int):
    """-> (grad_y_perm with NaN in rows no slot points at, grad_w)."""
    gy, yp = np.asarray(grad_y, np.float64), np.asarray(y_perm, np.float64)
    T = gy.shape[0]
    grad_rows = np.full(yp.shape, np.nan)
    grad_w = np.zeros((T, k))
    for t in range(T):
        for s in range(k):
            r = int(row_of[t * k + s])
            if r >= 0:
                grad_rows[r] = w[t, s] * gy[t]
                grad_w[t, s] = float(gy[t] @ yp[r])
    return grad_rows, grad_w


def adapter_delta(x, adapter, expert, a, b, scale) -> np.ndarray:
    """delta[row] = scale[n] B[n, e] (A[n, e] x[row]) with n the row's adapter
    (outside [0, N): zero) and e its expert."""
    x = np.asarray(x, np.float64)
    N = a.shape[0]
    out = np.zeros((x.shape[0], b.shape[2]))
    for r in range(x.shape[0]):
        n, e = int(adapter[r]), int(expert[r])
        if 0 <= n < N:
            out[r] = float(scale[n]) * (np.asarray(b[n, e], np.float64) @ (np.asarray(a[n, e], np.float64) @ x[r]))
    return out


def adapter_gate_up(x, adapter, expert, a, b, scale, pre, act: int) -> np.ndarray:
    v = np.asarray(pre, np.float64) + adapter_delta(x, adapter, expert, a, b, scale)
    if act == ACT_SWIGLU:
        f = v.shape[1] // 2
        return silu(v[:, :f]) * v[:, f:]
    return gelu(v)


def adapter_down(x, adapter, expert, a, b, scale, base) -> np.ndarray:
    return np.asarray(base, np.float64) + adapter_delta(x, adapter, expert, a, b, scale)
