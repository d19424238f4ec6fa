"""The 8-bit decode where values are extreme: large and tiny scales, gates of any sign, numbers
that are not finite in the live chunk, both forms of the call (one workgroup a row, and the split
one that few rows with a long cache take) on the same inputs."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import host, note
from test_gpu_cache8 import EPS, check_decode, hla, make_cache, rnd, row_cache, token

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("n_cap", [12, 130])
@pytest.mark.parametrize("sa,g", [(1.0, 1.0), (1e-3, 1.0), (2.0 ** -90, 0.5), (0.0, 1.0)], ids=str)
def test_scales_of_any_size(fmt, n_cap, sa, g):
    """Maps far from the identity (a chunk multiplies |z| by up to a few hundred: the fixed-point
    terms then need z's own maximum), near it, and equal to it.  The reference is the same chain in
    float64, and the bound follows the magnitudes through it."""
    note(f"cache8 scales {fmt} {n_cap} {sa} {g}")
    h = hla()
    dk, dv, n = 64, 64, 12
    c = make_cache(h, 1, 2, n_cap, dk, dv, 0, fmt, 201)
    c.count.fill_(n)
    c.scale[..., 0] = sa
    top = float(np.abs(host(c.maps.float())).max())
    (q, k, v), gates, S, A = token(1, 2, dk, dv, "f32", False, 202)
    S0, A0 = host(S), host(A)
    gi = torch.full((1, 2, n_cap), g, device="cuda")
    o = host(h.gdn_decode8(q, k, v, *gates, S, A, c, gates_in=gi, tau=0.0))
    for hh in range(2):
        cA, cB, _ = row_cache(c, 0, hh)
        beta, alpha = (float(x[0, hh]) for x in gates)
        lin = alpha * (np.eye(dk) - beta * np.outer(host(k)[0, hh], host(k)[0, hh]))
        B = S0[0, hh].T @ lin + beta * np.outer(host(v)[0, hh], host(k)[0, hh])
        z = A0[0, hh].T @ lin @ host(q)[0, hh]
        ref = B @ host(q)[0, hh]
        # each step's own rounding, (dk + 8) EPS of its sums of magnitudes (fixed point rounds z to
        # 2^-23 of its largest value), carried on by the chunks behind it
        err = (dk + 8) * EPS * (np.abs(B) @ np.abs(host(q)[0, hh]))
        ez = (dk + 8) * 4 * EPS * np.max(np.abs(z)) * np.ones(dk)
        for j in reversed(range(n)):
            E = cA[j] - np.eye(dk)
            zin = np.abs(z) + np.max(np.abs(z))
            ref = ref + g * cB[j] @ z
            err = err + g * np.abs(cB[j]) @ ez + (dk + 8) * 4 * EPS * g * (np.abs(cB[j]) @ zin) + EPS * np.abs(ref)
            ez = ez + g * np.abs(E) @ ez + (dk + 8) * 4 * EPS * (g * np.abs(E) @ zin + zin)
            z = z + g * E @ z
        assert np.all(np.isfinite(ref)) and top > 0
        assert np.all(np.abs(o[0, hh] - ref) <= err), (np.max(np.abs(o[0, hh] - ref)), np.max(err))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("n_cap", [20, 200])
def test_gates_of_any_sign(fmt, n_cap):
    note(f"cache8 signed gates {fmt} {n_cap}")
    h = hla()
    c = make_cache(h, 1, 3, n_cap, 128, 64, 0, fmt, 211)
    c.count.fill_(n_cap)
    c.count[0, 1] = n_cap - 7
    randn, _ = rnd(212)
    gi = randn(1, 3, n_cap) * 0.1
    check_decode(h, c, *token(1, 3, 128, 64, "bf16", False, 213), gates_in=gi, tau=-0.05)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("n_cap", [20, 200])
@pytest.mark.parametrize("what", ["q", "At", "S", "map"])
def test_not_finite_is_not_hidden(fmt, n_cap, what):
    """A NaN or an infinity that enters a row reaches that row's output and no other's."""
    note(f"cache8 not finite {fmt} {n_cap} {what}")
    if what == "map" and fmt == "int8":
        return  # no stored byte is not a number
    h = hla()
    c = make_cache(h, 1, 3, n_cap, 64, 128, 0, fmt, 221)
    c.count.fill_(n_cap)
    tok, gates, S, A = token(1, 3, 64, 128, "f32", False, 222)
    gi = torch.full((1, 3, n_cap), 0.3, device="cuda")
    clean = host(h.gdn_decode8(*tok, *gates, S.clone(), A.clone(), c, gates_in=gi))
    assert np.all(np.isfinite(clean))
    if what == "q":
        tok[0][0, 1, 5] = float("inf")
    elif what == "At":
        A[0, 1, 3, 7] = float("nan")
    elif what == "S":
        S[0, 1, 3, 7] = float("inf")
    else:
        c.maps.view(torch.uint8)[0, 1, int(c.order[0, 1, n_cap - 2]), 3, 9] = 0x7F
    o = host(h.gdn_decode8(*tok, *gates, S, A, c, gates_in=gi))
    assert np.array_equal(o[0, [0, 2]], clean[0, [0, 2]])
    if what == "S":
        assert not np.isfinite(o[0, 1]).all()
    else:
        assert not np.isfinite(o[0, 1]).any()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
def test_both_forms_on_the_same_rows(fmt, dk, dv):
    """Rows of a large batch (one workgroup a row) against the same rows as a small one (split)."""
    note(f"cache8 both forms {fmt} {dk}")
    h = hla()
    n_cap, H = 150, 2
    big = make_cache(h, 130, H, n_cap, dk, dv, 3, fmt, 231)
    _, rand = rnd(232)
    big.count.copy_((rand(130, H) * (n_cap + 1)).to(torch.int32).clamp(max=n_cap))
    big.count[:2] = torch.tensor([[n_cap, 40], [0, 63]], dtype=torch.int32)
    tok, gates, S, A = token(130, H, dk, dv, "bf16", False, 233)
    cut = lambda t: t[:2].contiguous().clone()  # noqa: E731
    small = h.Cache8(*(cut(t.view(torch.uint8)).view(t.dtype) if t.element_size() == 1 else cut(t)
                       for t in (big.maps, big.reps, big.scale, big.order, big.count, big.weight)))
    assert h.cache8_workspace_bytes(big) == 0 and h.cache8_workspace_bytes(small) > 0
    St, At = cut(S), cut(A)
    gb, gs = torch.empty(130, H, n_cap, device="cuda"), torch.empty(2, H, n_cap, device="cuda")
    ob = h.gdn_decode8(*tok, *gates, S, A, big, gates_out=gb)
    os_ = h.gdn_decode8(*(cut(t) for t in tok), *(cut(t) for t in gates), St, At, small, gates_out=gs)
    # two roundings of the same sums (see check_decode), in each form
    tol = 4 * (n_cap + 2) * (dk + 8) * EPS
    for a, b in ((ob, os_), (S, St), (A, At), (gb, gs), (big.weight, small.weight)):
        a, b = host(a[:2]), host(b)
        assert np.max(np.abs(a - b)) <= tol * max(1.0, np.max(np.abs(a)))


@pytest.mark.parametrize("n_cap", [20, 200])
def test_z_at_the_end_of_its_range(n_cap):
    """int8 chunks hold z below 2^127: just below, o is right; from there on it is NaN, not wrong."""
    note(f"cache8 largest z {n_cap}")
    h = hla()
    for zmax, fits in ((1.5 * 2.0 ** 126, True), (1.5 * 2.0 ** 127, False)):
        c = make_cache(h, 1, 1, n_cap, 64, 64, 0, "int8", 231)
        c.count.fill_(n_cap)
        c.scale[..., 0] = 0.0  # A = I: z stays as it enters
        c.scale[..., 1] = 2.0 ** -20
        zero, one = torch.zeros(1, 1, 64, device="cuda"), torch.ones(1, 1, device="cuda")
        q = zero.clone()
        q[..., 3] = 1.0
        S, A = torch.zeros(1, 1, 64, 64, device="cuda"), torch.zeros(1, 1, 64, 64, device="cuda")
        A[0, 0, 3, 5] = zmax  # z = zmax e_5
        gi = torch.full((1, 1, n_cap), 0.0, device="cuda")
        gi[..., n_cap // 2] = 1.0
        o = host(h.gdn_decode8(q, zero, zero, 0 * one, one, S, A, c, gates_in=gi, tau=0.5))[0, 0]
        if fits:
            ref = row_cache(c, 0, 0)[1][n_cap // 2][:, 5] * zmax
            assert np.all(np.abs(o - ref) <= 4 * EPS * np.abs(ref))
        else:
            assert np.isnan(o).all()


@pytest.mark.parametrize("n_cap", [30, 300])
def test_same_bits_every_time(n_cap):
    """Two equal calls give equal bits (fixed orders of summation in both forms)."""
    note(f"cache8 twice {n_cap}")
    h = hla()
    outs = []
    for _ in range(2):
        c = make_cache(h, 1, 4, n_cap, 128, 128, 5, "e4m3", 241)
        c.count.fill_(n_cap)
        tok, gates, S, A = token(1, 4, 128, 128, "bf16", True, 242)
        gout = torch.empty(1, 4, n_cap, device="cuda")
        o = h.gdn2_decode8(*tok, *gates, S, A, c, gates_out=gout)
        outs.append([t.clone() for t in (o, S, A, gout, c.weight)])
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_largest_representative_count():
    note("cache8 256 representatives")
    h = hla()
    for n_cap in (3, 70):
        c = make_cache(h, 1, 2, n_cap, 128, 64, 256, "int8", 251)
        c.count.fill_(n_cap)
        check_decode(h, c, *token(1, 2, 128, 64, "bf16", False, 252))
