"""Oracle of the 8-bit chunk cache: stored values, weights and eviction, one row at a time.

The stored formats are stated by their value sets: int8 the integers -127 .. 127, e4m3 the
numbers (-1)^s 2^(e-7) (1 + m/8) (e = 1 .. 15, without the NaN at e = 15, m = 7) and
(-1)^s 2^-6 m/8.  A block is multiplied by (1 / max) top in float32 (the definition's own
roundings) and each product goes to the nearest value of the set, ties to the even code.
"""
import numpy as np

TOP = {"int8": 127.0, "e4m3": 448.0}


def e4m3_values() -> np.ndarray:
    """The non-negative values by code 0 .. 126."""
    code = np.arange(127)
    e, m = code >> 3, code & 7
    return np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * 2.0 ** (e - 7.0))


def quantise(X, fmt):
    """(stored values as float64, scale) of one block X (float32 values)."""
    X = np.asarray(X, np.float32)
    m = np.float32(np.max(np.abs(X))) if X.size else np.float32(0)
    top = np.float32(TOP[fmt])
    if not np.all(np.isfinite(X)):
        return np.zeros(X.shape), float("nan")
    if not m >= np.float32(2.0 ** -100):
        return np.zeros(X.shape), 0.0
    y = (X * (np.float32(1) / m * top)).astype(np.float64)
    if fmt == "int8":
        return np.clip(np.rint(y), -127, 127), float(m * (np.float32(1) / top))
    values = e4m3_values()
    mag = np.minimum(np.abs(y), values[-1])
    hi = np.clip(np.searchsorted(values, mag), 1, len(values) - 1)
    lo = hi - 1
    up = (mag - values[lo] > values[hi] - mag) | ((mag - values[lo] == values[hi] - mag) & (hi % 2 == 0))
    return np.where(up, values[hi], values[lo]) * np.where(np.signbit(y), -1.0, 1.0), float(m * (np.float32(1) / top))


def gate_weights(gates, tau, n):
    """[N] weights of one row's gate matrix [N, N] with n valid chunks."""
    w = np.zeros(gates.shape[0])
    for j in range(n):
        for i in range(j + 1, n):
            g = np.float32(gates[i, j])
            if g >= np.float32(tau):
                w[j] += min(max(float(g), 0.0), 1.0)
    return w


def evict(weight, order, count, budget, n_recent):
    """(order, weight, count) of one row after the cut to `budget`."""
    n = len(weight)
    held = min(max(int(count), 0), n)
    gone = []
    if held > budget:
        lightness = [(-np.inf if np.isnan(weight[p]) else float(weight[p]), not np.isnan(weight[p]), p)
                     for p in range(held - n_recent)]
        gone = sorted(p for _, _, p in sorted(lightness)[:held - budget])
    kept = [p for p in range(held) if p not in set(gone)]
    out = np.zeros(n, np.float32)
    out[:len(kept)] = weight[kept]
    return order[kept + gone + list(range(held, n))], out, len(kept)
