"""The 8-bit decode against float64 to the precision of its arithmetic: bounds of a few float32
roundings (cache8_bounds, where a host test shows that a term or a chunk left out exceeds them),
for the form with one workgroup a row and for the split form."""
import numpy as np
import pytest
import torch

import cache8_bounds as cb
from gated_deltanet_hybrid_amd import inputs
from gpu_util import host, note, token_tensors
from test_gpu_cache8 import hla, make_cache, rnd, token, values

pytestmark = pytest.mark.gpu
EPS = cb.EPS


def check_close(h, c, tok, gates, S, A, gates_in=None, tau=1e-3, rows=None, seg=None):
    """One step; every row (or `rows`) within the bounds of cache8_bounds.  The chain's reference
    takes the gates that the step reports, which are checked by themselves.  ``seg``: bounds
    through segments of that many positions.  Returns the largest error over its tolerance."""
    q, k, v = tok
    S0, A0 = host(S), host(A)
    w0 = None if c.weight is None else host(c.weight)
    gout = torch.full((c.Bs, c.H, c.n_cap), float("nan"), device="cuda")
    fn = h.gdn2_decode8 if len(gates) == 3 else h.gdn_decode8
    o = host(fn(q, k, v, *gates, S, A, c, gates_in=gates_in, tau=tau, gates_out=gout))
    fmt = "int8" if c.maps.dtype == torch.int8 else "e4m3"
    rep32, S1, A1 = gout.cpu().numpy(), host(S), host(A)
    worst = 0.0
    for b, hh in rows or [(b, hh) for b in range(c.Bs) for hh in range(c.H)]:
        n = min(max(int(c.count[b, hh]), 0), c.n_cap)
        slots = c.order[b, hh, :n].long().clamp(0, c.n_cap - 1)
        m = values(c.maps[b, hh].view(torch.uint8)[slots].view(c.maps.dtype))
        sc = c.scale[b, hh][slots].cpu().numpy().astype(np.float64)
        tk = [host(x)[b, hh] for x in (q, k, v)]
        gt = [host(x)[b, hh] for x in gates]
        g = rep32[b, hh]
        assert np.all(g[n:] == 0.0), f"row {b},{hh}: gates behind the last chunk"
        if gates_in is not None:
            assert np.array_equal(g[:n], gates_in[b, hh, :n].cpu().numpy(), equal_nan=True)
        elif n:
            reps = values(c.reps[b, hh].view(torch.uint8)[slots].view(c.reps.dtype))
            for j in range(n):
                want, tol = cb.gate(tk[0], reps[j], sc[j, 2], fmt)
                assert abs(float(g[j]) - want) <= tol, f"row {b},{hh}: gate {j} is {g[j]}, not {want} +- {tol:.1e}"
        ghat = np.where(g[:n] >= np.float32(tau), g[:n], np.float32(0)).astype(np.float64)
        ref, tol = cb.chain(*tk, gt, S0[b, hh], A0[b, hh], m[:, :c.dk], m[:, c.dk:], sc[:, 0], sc[:, 1], ghat, fmt, seg)
        ratio = float(np.max(np.abs(o[b, hh] - ref) / tol))
        assert ratio <= 1.0, f"row {b},{hh}: n={n}: o is off by {ratio:.2f} tolerances"
        worst = max(worst, ratio)
        a, e, w = cb.token_rows(*tk, gt)
        for got, mat, ww in ((S1, S0, w), (A1, A0, None)):
            new, lim = cb.live_after(mat[b, hh], tk[1], a, e, ww)
            assert np.all(np.abs(got[b, hh] - new) <= lim + 2.0 ** -149), f"row {b},{hh}: live matrix"
        if w0 is not None:
            got = host(c.weight)[b, hh]
            want = w0[b, hh, :n] + np.clip(ghat, 0.0, 1.0)
            assert np.all(np.abs(got[:n] - want) <= EPS * np.abs(want)), f"row {b},{hh}: weights"
            assert np.array_equal(got[n:], w0[b, hh, n:])
    return worst


WHOLE = [  # fmt, dtype, dk, dv, Bs, H, n_cap, n_rep, gdn2
    ("int8", "bf16", 128, 128, 2, 3, 9, 2, False),
    ("e4m3", "bf16", 128, 128, 2, 3, 9, 64, True),
    ("int8", "f32", 64, 128, 1, 5, 17, 1, True),
    ("e4m3", "f32", 128, 64, 3, 2, 33, 5, False),
    ("int8", "bf16", 64, 64, 1, 3, 50, 17, True),
    ("e4m3", "f32", 64, 64, 2, 2, 16, 33, False),
    ("int8", "f32", 128, 64, 1, 2, 3, 256, False),
    ("e4m3", "bf16", 64, 128, 1, 1, 1, 3, True),
]
SPLIT = [
    ("int8", "bf16", 128, 128, 1, 3, 130, 2, False),
    ("e4m3", "f32", 128, 64, 1, 2, 200, 5, True),
    ("int8", "f32", 64, 64, 2, 2, 200, 3, True),
    ("e4m3", "bf16", 64, 128, 1, 3, 150, 40, False),
    ("int8", "bf16", 64, 128, 1, 1, 1024, 2, False),
    ("e4m3", "f32", 128, 128, 1, 1, 520, 1, False),
]


@pytest.mark.parametrize("case", WHOLE + SPLIT, ids=str)
@pytest.mark.parametrize("given", [False, True], ids=["scored", "given"])
def test_decode_to_rounding(case, given):
    fmt, dtype, dk, dv, Bs, H, n_cap, n_rep, gdn2 = case
    note(f"cache8 precision {case} {given}")
    h = hla()
    c = make_cache(h, Bs, H, n_cap, dk, dv, n_rep, fmt, 401)
    c.count.fill_(n_cap)
    if n_cap > 1:
        c.count[-1, -1] = n_cap - 1
    assert (h.cache8_workspace_bytes(c) > 0) == (case in SPLIT)
    gi = None
    if given:
        _, rand = rnd(402)
        gi = 0.05 + 0.9 * rand(Bs, H, n_cap)
    note(f"  worst {check_close(h, c, *token(Bs, H, dk, dv, dtype, gdn2, 403), gates_in=gi):.3f}")


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_many_rows_to_rounding(fmt):
    """More rows than the split form takes, every length: sampled rows."""
    note(f"cache8 precision many rows {fmt}")
    h = hla()
    Bs, H, n_cap, dk, dv = 90, 3, 100, 64, 64
    c = make_cache(h, Bs, H, n_cap, dk, dv, 4, fmt, 411)
    c.count.copy_((torch.arange(Bs * H, device="cuda") * 37 % (n_cap + 1)).view(Bs, H).to(torch.int32))
    assert h.cache8_workspace_bytes(c) == 0
    rows = [(b, b % H) for b in range(0, Bs, 3)]
    note(f"  worst {check_close(h, c, *token(Bs, H, dk, dv, 'bf16', False, 412), rows=rows):.3f}")


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dk", [64, 128])
def test_split_at_its_borders(fmt, dk):
    """Lengths on both sides of one segment, of a segment's end and of the full cache, in one call."""
    note(f"cache8 split borders {fmt} {dk}")
    h = hla()
    held = [0, 1, 63, 64, 65, 71, 72, 73, 128, 135, 136, 137, 199, 200]
    c = make_cache(h, 1, len(held), 200, dk, 64, 2, fmt, 421)
    c.count.copy_(torch.tensor([held], dtype=torch.int32))
    assert h.cache8_workspace_bytes(c) > 0
    note(f"  worst {check_close(h, c, *token(1, len(held), dk, 64, 'f32', False, 422)):.3f}")


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_both_forms_to_rounding(fmt):
    """The same rows in a large batch (one workgroup a row) and alone (split): each within the bounds,
    the live matrices and the gates equal to a rounding of the same sums."""
    note(f"cache8 both forms to rounding {fmt}")
    h = hla()
    n_cap, H, Bs = 150, 2, 130
    big = make_cache(h, Bs, H, n_cap, 64, 64, 3, fmt, 431)
    big.count.fill_(n_cap)
    big.count[1] = torch.tensor([40, 63], dtype=torch.int32)
    tok, gates, S, A = token(Bs, H, 64, 64, "bf16", False, 432)
    part = lambda t: t[:2].contiguous().clone()  # noqa: E731
    small = h.Cache8(*(part(t.view(torch.uint8)).view(t.dtype) if t.element_size() == 1 else part(t)
                       for t in (big.maps, big.reps, big.scale, big.order, big.count, big.weight)))
    assert h.cache8_workspace_bytes(big) == 0 and h.cache8_workspace_bytes(small) > 0
    rows = [(b, hh) for b in range(2) for hh in range(H)]
    St, At = part(S), part(A)
    check_close(h, big, tok, gates, S, A, rows=rows)
    check_close(h, small, [part(t) for t in tok], [part(t) for t in gates], St, At)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("alpha_mode", ["slow", "config"])
@pytest.mark.parametrize("n,dk,dv", [(1, 128, 128), (20, 64, 128), (100, 128, 64)], ids=str)
def test_what_eight_bits_cost(fmt, alpha_mode, n, dk, dv):
    """A prompt's chunks in the cache against the same decode over their unquantised maps: within what
    the stored numbers' roundings explain (the float32 arithmetic is three orders below)."""
    note(f"cache8 cost {fmt} {alpha_mode} {n} {dk} {dv}")
    h = hla()
    H = 2
    x = inputs.gen_tokens(1, 64 * n, H, dk, dv, dtype="f32", seed=441, alpha_mode=alpha_mode)
    _, k, v, beta, alpha = token_tensors(x)
    At, Bc = h.chunk_transitions(k, v, beta, alpha)
    c = h.cache8_alloc(1, H, n, dk, dv, 0, fmt)
    h.cache8_append(c, At, Bc)
    tok, gates, _, _ = token(1, H, dk, dv, "f32", False, 442)
    S, A = torch.zeros(1, H, dk, dv, device="cuda"), torch.eye(dk, device="cuda").repeat(1, H, 1, 1)
    S0, A0 = host(S), host(A)
    gi = 0.1 + 0.8 * rnd(443)[1](1, H, n)
    o = host(h.gdn_decode8(*tok, *gates, S, A, c, gates_in=gi))
    for hh in range(H):
        maps = [host(t)[0, hh].transpose(0, 2, 1) for t in (At, Bc)]
        tk, gt = [host(t)[0, hh] for t in tok], [host(t)[0, hh] for t in gates]
        ref, tol = cb.unquantised(*tk, gt, S0[0, hh], A0[0, hh], *maps, host(gi)[0, hh], fmt)
        past = ref - cb.live(S0[0, hh], tk[0], tk[1], *cb.token_rows(*tk, gt))[0]
        off = o[0, hh] - ref
        assert np.all(np.abs(off) <= tol + 1e-5 * np.max(np.abs(ref))), float(np.max(np.abs(off) / tol))
        share = np.linalg.norm(off) / np.linalg.norm(past)
        note(f"  {share:.4f} of the past's share, {float(np.max(np.abs(off) / tol)):.2f} of the bound")
