"""The decode step over the 8-bit chunk cache in float64, one row at a time, with the rounding
that its float32 arithmetic may leave -- a bound close enough to see a term left out.

Every rounding is taken as an independent error of at most half a step (EPS relative) of what is
rounded, and its variance is carried along the chain: a sum of m products, added in any order, has
partial sums of about sqrt(k) of a term's size after k of them, so its roundings' variance is at
most EPS^2 (m / 2) sum t_i^2.  The tolerance is six standard deviations: over the some thousand
outputs of a case an independent error passes it with probability 1e-5 or less, and the variances
themselves are upper bounds (real sums are trees, and errors of half a step are the largest).
What a chunk's map does to z is counted once for the sum and once for the addition to z; a segment
of the split form adds one more pass over z for at least eight chunks, 24 additions that hold z
itself, hence the 4 in ``chain``."""
import numpy as np

EPS = 2.0 ** -24
SIGMAS = 6.0


def live(mat, q, k, a, e, w):
    """(mat after the token read with q, its variance) by column: mat [dk, W], w [W] or None."""
    h = len(q) / 2
    u, aq = (a * k) @ mat, (a * q) @ mat
    qe, qk = q @ e, q @ k
    ww = np.zeros(mat.shape[1]) if w is None else w
    var = h * (((a * q)[:, None] * mat) ** 2).sum(0) + h * qe ** 2 * (((a * k)[:, None] * mat) ** 2).sum(0)
    var += h * u ** 2 * ((q * e) ** 2).sum() + h * ww ** 2 * ((q * k) ** 2).sum()
    var += 4 * (aq ** 2 + (qe * u) ** 2 + (qk * ww) ** 2)
    return aq - qe * u + qk * ww, EPS ** 2 * var


def live_after(mat, k, a, e, w):
    """The live matrix after the token, and its tolerance."""
    u = (a * k) @ mat
    add = 0.0 if w is None else np.outer(k, w)
    new = a[:, None] * mat - np.outer(e, u) + add
    var = len(k) / 2 * np.outer(e ** 2, ((a * k)[:, None] ** 2 * mat ** 2).sum(0))
    var = var + 4 * ((a[:, None] * mat) ** 2 + np.outer(e, u) ** 2 + add ** 2)
    return new, SIGMAS * EPS * np.sqrt(var)


def token_rows(q, k, v, gates):
    """(a, e, w) of the live update: gates (beta, alpha) or (a, b, w)."""
    if len(gates) == 3:
        return gates[0], gates[1] * k, gates[2] * v
    beta, alpha = gates
    return np.full(len(k), float(alpha)), beta * k, beta * v


def _grown(x2, var, ca, E):
    """Variance of (I + ca E) x, of variance ``var`` and square ``x2``: what ``var`` becomes, and the
    roundings of the sum and of its addition."""
    diag, E2 = np.diagonal(E) * ca, ca ** 2 * E ** 2
    own = np.reshape((1 + diag) ** 2 - diag ** 2, (-1,) + (1,) * (var.ndim - 1))
    return own * var + E2 @ var + EPS ** 2 * (len(E) / 2) * (E2 @ x2)


def chain(q, k, v, gates, S, A, E8, B8, sa, sb, ghat, fmt, seg=None):
    """(o, tolerance) of one row.  S [dk, dv] and A [dk, dk] before the step (state orientation),
    E8 [n, dk, dk] and B8 [n, dv, dk] the stored numbers with their scales, ghat the gates after
    the threshold, in time order.  With ``seg`` the bound is the split form's: z passes from one
    segment of that many positions to the next through the segment's composed map P (the same z but
    for rounding; far from the identity P's own roundings count for more than the chain's)."""
    dk = len(q)
    h = dk / 2
    a, e, w = token_rows(q, k, v, gates)
    o, vo = live(S, q, k, a, e, w)
    z, vz = live(A, q, k, a, e, None)
    past = np.zeros_like(o)
    fixed = 1.0  # int8: the bound of |z| that the operand in use was written for, over its largest |z|
    P, vP, z0, v0 = np.eye(dk), np.zeros((dk, dk)), z, vz
    for j in reversed(range(len(ghat))):
        if ghat[j] != 0.0:
            step = (2.0 ** -29 * fixed * np.max(np.abs(z))) ** 2 if fmt == "int8" else 0.0
            ca, cb = ghat[j] * sa[j], ghat[j] * sb[j]
            B2, E2 = B8[j] ** 2, E8[j] ** 2
            y = cb * (B8[j] @ z)
            past = past + y
            vo = vo + cb ** 2 * (B2 @ vz) + EPS ** 2 * (h * cb ** 2 * (B2 @ z ** 2) + 2 * past ** 2 + 4 * y ** 2)
            vo = vo + cb ** 2 * step * B2.sum(1)
            d = ca * (E8[j] @ z)
            vz = _grown(z ** 2, vz, ca, E8[j]) + ca ** 2 * step * E2.sum(1) + EPS ** 2 * 4 * ((z + d) ** 2 + d ** 2)
            z = z + d
            fixed = min(1.0 + abs(ca) * 128 * dk, 128.0)
            if seg:
                D = ca * (E8[j] @ P)
                vP = _grown(P ** 2, vP, ca, E8[j]) + EPS ** 2 * 4 * ((P + D) ** 2 + D ** 2)
                P = P + D
        if seg and j % seg == 0:
            vz = P ** 2 @ v0 + vP @ z0 ** 2 + EPS ** 2 * h * (P ** 2 @ z0 ** 2)
            P, vP, z0, v0, fixed = np.eye(dk), np.zeros((dk, dk)), z, vz, 1.0
    out = o + past
    return out, SIGMAS * np.sqrt(vo + EPS ** 2 * 2 * out ** 2)


def gate(q, R8, scale, fmt):
    """(gate, tolerance) of one chunk scored by stored representatives [n_rep, dk]."""
    dk = len(q)
    f = scale / np.sqrt(dk)
    s = (R8 @ q) * f
    vs = EPS ** 2 * (dk / 2 * f ** 2 * (R8 ** 2 @ q ** 2) + 4 * s ** 2)
    if fmt == "int8":  # q rounded against its largest value
        vs = vs + (2.0 ** -29 * np.max(np.abs(q)) * f) ** 2 * (R8 ** 2).sum(1)
    m = s.max()
    p = np.exp(s - m)
    logit = m + np.log(p.mean())
    share = p / p.sum()
    # the exponentials' and their sum's own roundings (relative to the sum, whose logarithm is taken:
    # a step or two each, the argument's 2 EPS |s - m| <= 2 EPS of the largest term), then of the logit
    var = (share ** 2 * vs).sum() + EPS ** 2 * (len(s) / 2 + 32 + 8 * logit ** 2)
    g = 1.0 / (1.0 + np.exp(-logit))
    return g, SIGMAS * np.sqrt((g * (1 - g)) ** 2 * var + EPS ** 2 * 16 * g ** 2)


def step_variance(X, fmt):
    """Variance of each number of a block that is stored in 8 bits: a rounding error spread evenly over
    a step of the stored value, in the block's own unit."""
    top = {"int8": 127.0, "e4m3": 448.0}[fmt]
    m = np.max(np.abs(X))
    if m == 0.0:
        return np.zeros(X.shape)
    y = np.abs(X) / m * top
    step = np.ones(X.shape) if fmt == "int8" else 2.0 ** (np.floor(np.log2(np.maximum(y, 2.0 ** -6))) - 3)
    return (step * m / top) ** 2 / 12


def unquantised(q, k, v, gates, S, A, cA, cB, ghat, fmt):
    """(o over the maps cA [n, dk, dk] and cB [n, dv, dk] as they were before they were stored in 8
    bits, what storing them may change o by: six standard deviations of the stored numbers' roundings,
    carried along the chain)."""
    a, e, w = token_rows(q, k, v, gates)
    o, _ = live(S, q, k, a, e, w)
    z, _ = live(A, q, k, a, e, None)
    vo, vz = np.zeros(len(o)), np.zeros(len(z))
    for j in reversed(range(len(ghat))):
        g, E = ghat[j], cA[j] - np.eye(len(q))
        o = o + g * (cB[j] @ z)
        vo = vo + g ** 2 * (cB[j] ** 2 @ vz + step_variance(cB[j], fmt) @ (z ** 2 + vz))
        vz = (1 + g * np.diagonal(E)) ** 2 * vz - (g * np.diagonal(E)) ** 2 * vz + g ** 2 * (
            E ** 2 @ vz + step_variance(E, fmt) @ (z ** 2 + vz))
        z = z + g * (E @ z)
    return o, SIGMAS * np.sqrt(vo)
