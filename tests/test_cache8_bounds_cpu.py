"""The bounds that the 8-bit decode is held to (cache8_bounds), on the host: the reference chain is
the oracle's step, numpy models of the kernels' arithmetic lie well inside the bounds, and the same
models with one term or one chunk left out lie outside (no GPU needed)."""
import math

import numpy as np
import pytest
import torch

import cache8_bounds as cb
import oracle

F32 = np.float32
SIZES = [(1, 128, 128), (9, 128, 128), (17, 64, 128), (70, 64, 64), (200, 128, 64), (1024, 64, 64)]


def row(n, dk, dv, fmt, seed):
    """One row as the GPU tests draw it: maps whose E has a spectral norm near 0.25, gates in (0, 1)."""
    r = np.random.default_rng(seed)
    f = lambda x: np.asarray(x, F32).astype(np.float64)  # noqa: E731
    top = {"int8": 127.0, "e4m3": 448.0}[fmt]
    m = np.clip(r.standard_normal((n, dk + dv, dk)) * 0.25 * top, -top, top).round()
    if fmt == "e4m3":
        m = torch.from_numpy(m).to(torch.float8_e4m3fn).double().numpy()
    sa, sb = f((0.5 + r.random(n)) / (2 * math.sqrt(dk) * top)), f((0.5 + r.random(n)) * 4 / top)
    k = r.standard_normal(dk)
    q, k, v = f(r.standard_normal(dk)), f(k / np.linalg.norm(k)), f(r.standard_normal(dv))
    S, A = f(r.standard_normal((dk, dv)) * 0.3), f(np.eye(dk) - 0.3 * r.random((dk, dk)) / math.sqrt(dk))
    return q, k, v, (float(f(r.random())), float(f(0.5 + 0.5 * r.random()))), S, A, m[:, :dk], m[:, dk:], sa, sb, \
        f(0.05 + 0.9 * r.random(n))


def cut(x):
    return (np.ascontiguousarray(x, F32).view(np.uint32) & np.uint32(0xFFFF0000)).view(F32)


def bf16_terms(x, keep):
    out, left = np.zeros(x.shape), np.asarray(x, F32)
    for _ in range(keep):
        out, left = out + cut(left), left - cut(left)
    return out


def fixed_bytes(x, bound, keep):
    """x against 2^e > bound as the `keep` upper ones of its four signed bytes."""
    e = math.frexp(bound)[1]
    F = np.trunc(x * 2.0 ** (30 - e)).astype(np.int64) + 0x808080
    out = (F >> 24) << 24
    for i in range(4 - keep, 3):
        out = out + ((F >> 8 * i & 255) - 128 << 8 * i)
    return out * 2.0 ** (e - 30)


def model(case, fmt, keep, skip=None, seg=None, keep_phi=3):
    """The chain in float32 with z as `keep` terms; with `seg` the linear parts of that many positions
    at a time composed first, each matrix as `keep_phi` bf16 terms in its products."""
    q, k, v, gates, S, A, E8, B8, sa, sb, g = case
    a, e, w = cb.token_rows(q, k, v, gates)
    o, z = cb.live(S, q, k, a, e, w)[0].astype(F32), cb.live(A, q, k, a, e, None)[0].astype(F32)
    ca, cbs = F32(g) * F32(sa), F32(g) * F32(sb)

    def segment(z, lo, hi):
        past, bound = np.zeros_like(o), np.abs(z).max()
        for j in reversed(range(lo, hi)):
            if j == skip:
                continue
            x = bf16_terms(z, keep) if fmt == "e4m3" else fixed_bytes(z.astype(np.float64), float(bound), keep)
            past = past + (cbs[j] * (B8[j] @ x)).astype(F32)
            factor = 1 + abs(ca[j]) * 128 * len(q)
            bound = np.abs(z).max() * factor
            z = z + (ca[j] * (E8[j] @ x)).astype(F32)
            bound = bound if factor <= 128 else np.abs(z).max()
        return past, z

    n = len(g)
    if seg is None:
        return o + segment(z, 0, n)[0]
    for lo in reversed(range(0, n, seg)):
        hi = min(lo + seg, n)
        o = o + segment(z, lo, hi)[0]
        P = np.eye(len(q), dtype=F32)
        for j in reversed(range(lo, hi)):
            P = P + ca[j] * (E8[j] @ bf16_terms(P, keep_phi)).astype(F32)
        z = (P.astype(np.float64) @ z).astype(F32)
    return o


@pytest.mark.parametrize("gdn2", [False, True])
def test_the_reference_is_the_oracles_step(gdn2):
    case = row(7, 64, 128, "int8", 1)
    q, k, v, gates, S, A, E8, B8, sa, sb, g = case
    g[2] = 0.0
    if gdn2:
        r = np.random.default_rng(2)
        gates = (r.random(64), r.random(64), r.random(128))
    step = oracle.gdn2_decode_step if gdn2 else oracle.decode_step
    cA, cB = np.eye(64) + E8 * sa[:, None, None], B8 * sb[:, None, None]
    ref = step(q, k, v, *gates, S.T, A.T, cA, cB, None, 1e-3, gates_in=g)
    o, tol = cb.chain(q, k, v, gates, S, A, E8, B8, sa, sb, g, "int8")
    assert np.max(np.abs(o - ref["o"])) <= 1e-12 * np.max(np.abs(o)) and np.all(tol > 0)
    a, e, w = cb.token_rows(q, k, v, gates)
    for mat, want, ww in ((S, ref["B_cur"].T, w), (A, ref["A_cur"].T, None)):
        new, tol = cb.live_after(mat, k, a, e, ww)
        assert np.max(np.abs(new - want)) <= 1e-13 * np.max(np.abs(want)) and np.all(tol[new != 0] > 0)
    R = np.random.default_rng(3).integers(-127, 128, (5, 64)).astype(float)
    got, _ = cb.gate(q, R, 0.01, "int8")
    assert abs(got - oracle.decode_step(q, k, v, 0.5, 0.5, S.T, A.T, cA[:1], cB[:1], 0.01 * R[None], 0.0)["gates"][0]) < 1e-14


def worst(case, fmt, *a, **kw):
    o, tol = cb.chain(*case, fmt)
    return np.max(np.abs(model(case, fmt, *a, **kw) - o) / tol)


@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("fmt,full", [("int8", 4), ("e4m3", 3)])
def test_lost_terms_and_chunks_are_seen(size, fmt, full):
    n, dk, dv = size
    case = row(n, dk, dv, fmt, n)
    assert worst(case, fmt, full) < 0.5
    assert worst(case, fmt, 2) > 2.0  # int8: the two lower bytes left out; e4m3: the third term
    assert worst(case, fmt, full, skip=int(np.argmin(case[-1]))) > 100.0  # the chunk of least weight
    if n > 64:
        assert worst(case, fmt, full, seg=8 if n <= 200 else 23) < 0.5
        assert worst(case, fmt, full, seg=8 if n <= 200 else 23, keep_phi=2) > 1.2


SCALES = [(1.0, [3, 40, 41, 42, 64, 96, 103, 129]), (2.0 ** -7, [0, 8, 15, 50, 51, 52, 53, 54, 55, 90, 127]),
          (1e-3, [5, 16, 23, 70, 71, 72, 100, 101, 120, 121, 122, 128]), (2.0 ** -90, [1, 30, 31, 32, 88, 129]),
          (0.0, [2, 9, 77, 78, 110])]


@pytest.mark.parametrize("sa,used", SCALES, ids=str)
@pytest.mark.parametrize("fmt,full", [("int8", 4), ("e4m3", 3)])
def test_lost_terms_are_seen_at_every_scale(sa, used, fmt, full):
    """Maps that multiply |z| by a few hundred down to the identity, few in use: the bound stays close
    to the output in both forms, and a lost term is outside it."""
    q, k, v, gates, S, A, E8, B8, _, sb, _ = row(130, 64, 64, fmt, 5)
    g = np.zeros(130)
    g[used] = 0.75
    case = (q, k, v, gates, S, A, E8, B8, np.full(130, float(F32(sa))), sb, g)
    for seg in (None, 8):
        o, tol = cb.chain(*case, fmt, seg=seg)
        assert np.max(tol) <= 2e-5 * np.max(np.abs(o))
        off = lambda keep, phi: np.max(np.abs(model(case, fmt, keep, seg=seg, keep_phi=phi) - o) / tol)  # noqa: E731
        assert off(full, 3) < 0.5 and off(2, 3) > 1.2
        if seg and sa in (1.0, 2.0 ** -7):
            assert off(full, 2) > 1.2
