"""The 8-bit chunk cache on the GPU against plain float64: the bytes and scales that append
stores, the decode step over any set of slots, the gate weights, eviction, and the calls as a
decoding program strings them together."""
import math

import numpy as np
import pytest
import torch

import oracle
import oracle.cache8 as o8
from gated_deltanet_hybrid_amd import inputs
from gpu_util import host, note, token_tensors

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24  # half a step of float32
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}
STORED = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def hla():
    from gated_deltanet_hybrid_amd import hla as h
    return h


def rnd(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (lambda *s: torch.randn(s, generator=g, device="cuda")), (lambda *s: torch.rand(s, generator=g, device="cuda"))


def values(t):
    """Stored numbers as float64 (8-bit floats go through float32 exactly)."""
    return t.float().cpu().numpy().astype(np.float64)


def make_cache(h, Bs, H, n_cap, dk, dv, n_rep, fmt, seed, weights=True):
    """A cache with every slot filled with contractions near the identity, in a shuffled order."""
    randn, rand = rnd(seed)
    c = h.cache8_alloc(Bs, H, n_cap, dk, dv, n_rep, fmt, weights=weights)
    top = o8.TOP[fmt]
    c.maps.copy_((randn(Bs, H, n_cap, dk + dv, dk) * 0.25 * top).clamp(-top, top).round().to(STORED[fmt]))
    if n_rep:
        c.reps.copy_((randn(Bs, H, n_cap, n_rep, dk) * 0.25 * top).clamp(-top, top).round().to(STORED[fmt]))
    # |E| entries ~ 0.25 top sA: a spectral norm near 0.25
    c.scale[..., 0] = (0.5 + rand(Bs, H, n_cap)) / (2 * math.sqrt(dk) * top)
    c.scale[..., 1] = (0.5 + rand(Bs, H, n_cap)) * 4 / top
    c.scale[..., 2] = (0.5 + rand(Bs, H, n_cap)) * 4 / top
    c.order.copy_(rand(Bs, H, n_cap).argsort(-1).to(torch.int32))
    if weights:
        c.weight.copy_(rand(Bs, H, n_cap))
    return c


def token(Bs, H, dk, dv, dtype, gdn2, seed):
    randn, rand = rnd(seed)
    q = randn(Bs, H, dk).to(TORCH[dtype])
    k = torch.nn.functional.normalize(randn(Bs, H, dk), dim=-1).to(TORCH[dtype])
    v = randn(Bs, H, dv).to(TORCH[dtype])
    gates = (0.5 + 0.5 * rand(Bs, H, dk), rand(Bs, H, dk), rand(Bs, H, dv)) if gdn2 else (rand(Bs, H), 0.5 + 0.5 * rand(Bs, H))
    S = randn(Bs, H, dk, dv) * 0.3
    A = torch.eye(dk, device="cuda") - 0.3 * rand(Bs, H, dk, dk) / math.sqrt(dk)
    return (q, k, v), gates, S, A


def row_cache(c, b, h):
    """(A, B, reps) of the held positions in time order, float64."""
    n = min(max(int(c.count[b, h]), 0), c.n_cap)
    slots = c.order[b, h, :n].long()
    m = values(c.maps[b, h].view(torch.uint8)[slots].view(c.maps.dtype))
    sc = c.scale[b, h, slots].cpu().numpy().astype(np.float64)
    A = np.eye(c.dk) + m[:, :c.dk] * sc[:, 0, None, None]
    B = m[:, c.dk:] * sc[:, 1, None, None]
    R = None
    if c.n_rep:
        R = values(c.reps[b, h].view(torch.uint8)[slots].view(c.maps.dtype)) * sc[:, 2, None, None]
    return A, B, R


def check_decode(h, c, tok, gates, S, A, gates_in=None, tau=1e-3):
    """One step, every row against the oracle on the values the cache stands for."""
    q, k, v = tok
    S0, A0 = host(S), host(A)
    w0 = None if c.weight is None else host(c.weight)
    gout = torch.full((c.Bs, c.H, c.n_cap), float("nan"), device="cuda")
    before = [t.clone() for t in (c.maps.view(torch.uint8), c.scale.view(torch.int32), c.order, c.count)]
    fn = h.gdn2_decode8 if len(gates) == 3 else h.gdn_decode8
    o = fn(q, k, v, *gates, S, A, c, gates_in=gates_in, tau=tau, gates_out=gout)
    torch.cuda.synchronize()
    for t, b in zip((c.maps.view(torch.uint8), c.scale.view(torch.int32), c.order, c.count), before):
        assert torch.equal(t, b), "the cache's contents changed"
    for b in range(c.Bs):
        for hh in range(c.H):
            cA, cB, R = row_cache(c, b, hh)
            n = len(cA)
            tk = [host(x)[b, hh] for x in (q, k, v)]
            gt = [host(x)[b, hh] for x in gates]
            gi = None if gates_in is None else host(gates_in)[b, hh]
            step = oracle.gdn2_decode_step if len(gates) == 3 else oracle.decode_step
            gt = gt if len(gates) == 3 else [float(x) for x in gt]
            ref = step(*tk, *gt, S0[b, hh].T, A0[b, hh].T, cA, cB, R, tau, gates_in=gi)
            # rounding, worst case: a dot product of dk terms is off by (dk + 4) EPS of the sum of
            # magnitudes; one live update and n composed chunks follow one another, and the norms
            # along them stay within twice the output's largest value
            scale = max(1.0, float(np.max(np.abs(ref["o"]))))
            tol = 2 * (n + 2) * (c.dk + 8) * EPS * scale
            err = np.max(np.abs(host(o)[b, hh] - ref["o"]))
            assert err <= tol, f"o row {b},{hh} n={n}: {err:.3e} > {tol:.3e}"
            lin = (c.dk + 8) * 4 * EPS
            assert np.max(np.abs(host(S)[b, hh] - ref["B_cur"].T)) <= lin * max(1.0, np.max(np.abs(ref["B_cur"])))
            assert np.max(np.abs(host(A)[b, hh] - ref["A_cur"].T)) <= lin * max(1.0, np.max(np.abs(ref["A_cur"])))
            g = host(gout)[b, hh]
            assert np.all(g[n:] == 0.0), "gates behind the last chunk"
            if gi is not None:
                assert np.array_equal(g[:n], gi[:n], equal_nan=True)
                gtol = 0.0
            elif n:
                # the logit is off by the score's rounding and a few steps of exp and log
                mag = np.abs(R) @ np.abs(tk[0]) / math.sqrt(c.dk)
                gtol = 0.25 * ((c.dk + 4) * EPS * np.max(mag) + 16 * EPS * (1 + np.max(np.abs(mag)))) + 4 * EPS
                assert np.max(np.abs(g[:n] - ref["gates"])) <= gtol
            if w0 is not None and n:
                want = w0[b, hh, :n] + np.clip(ref["ghat"], 0.0, 1.0)
                assert np.max(np.abs(host(c.weight)[b, hh, :n] - want)) <= gtol + 2 * EPS * np.max(want)
            if w0 is not None:
                assert np.array_equal(host(c.weight)[b, hh, n:], w0[b, hh, n:])
    return o


# ------------------------------------------------------------------------------- decode
CASES = [  # fmt, dtype, dk, dv, Bs, H, n_cap, n_rep, gdn2
    ("int8", "bf16", 128, 128, 2, 2, 9, 2, False),
    ("e4m3", "bf16", 128, 128, 2, 2, 9, 64, True),
    ("int8", "f32", 64, 128, 1, 5, 17, 1, True),
    ("e4m3", "f32", 128, 64, 3, 1, 33, 5, False),
    ("int8", "bf16", 64, 64, 1, 3, 70, 17, False),
    ("e4m3", "f32", 64, 64, 2, 2, 16, 33, True),
    ("int8", "f32", 128, 128, 1, 2, 5, 130, False),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_decode_parity(case):
    fmt, dtype, dk, dv, Bs, H, n_cap, n_rep, gdn2 = case
    note(f"decode8 {case}")
    h = hla()
    c = make_cache(h, Bs, H, n_cap, dk, dv, n_rep, fmt, 1)
    c.count.copy_(torch.randint(0, n_cap + 1, (Bs, H), generator=torch.Generator().manual_seed(2)).to(torch.int32))
    c.count.view(-1)[0] = n_cap
    check_decode(h, c, *token(Bs, H, dk, dv, dtype, gdn2, 3))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_decode_counts_and_masks(fmt):
    """Rows with nothing: no chunk, counts out of range, every gate below tau, NaN and infinite
    gates; bytes that no held position names (0xFF is e4m3's NaN) stay unread."""
    note(f"decode8 counts and masks {fmt}")
    h = hla()
    Bs, H, n_cap, dk, dv = 1, 8, 12, 64, 128
    c = make_cache(h, Bs, H, n_cap, dk, dv, 3, fmt, 11)
    c.count.copy_(torch.tensor([[0, 1, 12, 7, 40, -3, 12, 5]], dtype=torch.int32))
    for hh in range(H):
        n = min(max(int(c.count[0, hh]), 0), n_cap)
        for p in range(n, n_cap):
            s = int(c.order[0, hh, p])
            c.maps.view(torch.uint8)[0, hh, s] = 0xFF
            c.reps.view(torch.uint8)[0, hh, s] = 0xFF
            c.scale[0, hh, s] = float("nan")
    tok, gates, S, A = token(Bs, H, dk, dv, "f32", False, 12)
    check_decode(h, c, tok, gates, S, A)
    check_decode(h, c, tok, gates, S, A, tau=1.5)  # above every gate
    _, rand = rnd(13)
    g = rand(Bs, H, n_cap)
    g[0, 2, ::2] = float("nan")
    g[0, 3] = -1.0
    g[0, 6] = 0.0
    for hh in range(H):
        g[0, hh, min(max(int(c.count[0, hh]), 0), n_cap):] = float("inf")
    check_decode(h, c, tok, gates, S, A, gates_in=g, tau=0.3)
    check_decode(h, c, tok, gates, S, A, gates_in=g, tau=0.0)
    check_decode(h, c, tok, gates, S, A, gates_in=g, tau=-float("inf"))


def test_decode_slot_out_of_range_is_read_as_the_last():
    note("decode8 slot out of range")
    h = hla()
    a, b = (make_cache(h, 1, 2, 6, 64, 64, 2, "int8", 21) for _ in range(2))
    for c in (a, b):
        c.count.fill_(6)
    a.order[0, :, 2] = 1 << 20
    a.order[0, 0, 4] = -7
    b.order[0, :, 2] = 5
    b.order[0, 0, 4] = 5
    outs = []
    for c in (a, b):
        tok, gates, S, A = token(1, 2, 64, 64, "bf16", False, 22)
        outs.append(hla().gdn_decode8(*tok, *gates, S, A, c))
    assert torch.equal(outs[0], outs[1])


@pytest.mark.parametrize("case", [("int8", "bf16", 128, 128, 1, 2, False), ("e4m3", "f32", 64, 64, 1, 1, True)], ids=str)
def test_decode_longest_cache(case):
    fmt, dtype, dk, dv, Bs, H, gdn2 = case
    note(f"decode8 longest cache {case}")
    h = hla()
    c = make_cache(h, Bs, H, 1024, dk, dv, 1, fmt, 31)
    c.count.fill_(1024)
    c.count[0, 0] = 1023
    _, rand = rnd(32)
    on = rand(Bs, H, 1024) < 0.5
    g = torch.where(on, 0.02 + 0.05 * rand(Bs, H, 1024), 0.0)  # every part of the chain reaches the output
    check_decode(h, c, *token(Bs, H, dk, dv, dtype, gdn2, 33), gates_in=g, tau=0.01)
    check_decode(h, c, *token(Bs, H, dk, dv, dtype, gdn2, 34))


@pytest.mark.parametrize("n_cap", [40, 200])
@pytest.mark.parametrize("rows", [(1, 1), (3, 7), (40, 16)], ids=str)
def test_decode_rows_and_lengths(rows, n_cap):
    """Few and many rows, short and long caches (whatever split the call takes), no weights and
    no gates asked for: the same outputs as the oracle on sampled rows."""
    note(f"decode8 rows {rows} n_cap {n_cap}")
    h = hla()
    Bs, H = rows
    dk, dv = 128, 64
    c = make_cache(h, Bs, H, n_cap, dk, dv, 4, "int8", 41, weights=False)
    _, rand = rnd(42)
    c.count.copy_((rand(Bs, H) * (n_cap + 1)).to(torch.int32).clamp(max=n_cap))
    c.count[-1, -1] = n_cap
    tok, gates, S, A = token(Bs, H, dk, dv, "bf16", False, 43)
    S0, A0 = host(S), host(A)
    o = host(h.gdn_decode8(*tok, *gates, S, A, c))
    for b, hh in {(0, 0), (Bs - 1, H - 1), (Bs // 2, H // 2)}:
        cA, cB, R = row_cache(c, b, hh)
        ref = oracle.decode_step(*(host(x)[b, hh] for x in tok), *(float(x[b, hh]) for x in gates), S0[b, hh].T,
                                 A0[b, hh].T, cA, cB, R, 1e-3)
        tol = 2 * (len(cA) + 2) * (dk + 8) * EPS * max(1.0, float(np.max(np.abs(ref["o"]))))
        assert np.max(np.abs(o[b, hh] - ref["o"])) <= tol


# ------------------------------------------------------------------------------- append
def check_slot(c, b, h, slot, At, Bc, reps, fmt):
    m = values(c.maps[b, h, slot].view(torch.uint8).view(c.maps.dtype))
    for k, (X, got) in enumerate(((At.T - np.eye(c.dk, dtype=np.float32), m[:c.dk]), (Bc.T, m[c.dk:]))):
        want, scale = o8.quantise(X, fmt)
        assert np.array_equal(got, want), f"stored values of part {k}"
        assert float(c.scale[b, h, slot, k]) == np.float32(scale)
    if c.n_rep:
        want, scale = o8.quantise(reps, fmt)
        assert np.array_equal(values(c.reps[b, h, slot]), want)
        assert float(c.scale[b, h, slot, 2]) == np.float32(scale)
    assert float(c.scale[b, h, slot, 3]) == 0.0


def f32s(t):
    return t.float().cpu().numpy()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype,dk,dv,n_rep", [("bf16", 128, 128, 3), ("f32", 128, 64, 64), ("bf16", 64, 128, 1),
                                               ("f32", 64, 64, 0), ("bf16", 128, 64, 17), ("f32", 128, 128, 2)])
def test_append_stores_the_nearest_values(fmt, dtype, dk, dv, n_rep):
    """Ragged counts, a source list with repeats, no room left, then a second append behind the
    first; what is not appended stays as it was."""
    note(f"append8 {fmt} {dtype} {dk} {dv} {n_rep}")
    h = hla()
    Bs, H, n_cap, L, n = 2, 3, 6, 5, 4
    randn, rand = rnd(51)
    c = h.cache8_alloc(Bs, H, n_cap, dk, dv, n_rep, fmt)
    c.maps.view(torch.uint8).fill_(7)
    c.order.copy_(rand(Bs, H, n_cap).argsort(-1).to(torch.int32))
    c.count.fill_(3)
    At = (torch.eye(dk, device="cuda") + randn(Bs, H, L, dk, dk) * 0.1).to(TORCH[dtype])
    Bc = (randn(Bs, H, L, dk, dv) * torch.exp(3 * randn(Bs, H, L, 1, 1))).to(TORCH[dtype])
    At[0, 0, 0] = torch.eye(dk, device="cuda")  # A - I = 0: scale 0
    Bc[0, 0, 1] = 2.0 ** -120
    reps = randn(Bs, n * max(n_rep, 1), H, dk).to(TORCH[dtype])
    src = torch.tensor([0, 1, 3, 1, 9], dtype=torch.int32, device="cuda").repeat(Bs, H, 1)
    n_new = torch.tensor([[4, 2, 9], [0, -1, 3]], dtype=torch.int32, device="cuda")
    win = rand(Bs, H, L)
    for reset, start in ((True, 0), (False, 3)):
        c.count.fill_(start if not reset else 5)
        order0, maps0, w0 = c.order.clone(), c.maps.view(torch.uint8).clone(), c.weight.clone()
        h.cache8_append(c, At, Bc, reps if n_rep else None, src=src, n_new=n_new, weight_in=win, reset=reset, n=n)
        torch.cuda.synchronize()
        for b in range(Bs):
            for hh in range(H):
                want = min(max(int(n_new[b, hh]), 0), n, n_cap - start)
                assert int(c.count[b, hh]) == start + want
                order = list(range(n_cap)) if reset else order0[b, hh].tolist()
                assert c.order[b, hh].tolist() == order
                touched = set()
                for i in range(want):
                    s, slot = min(int(src[b, hh, i]), n - 1), order[start + i]
                    touched.add(slot)
                    R = None if not n_rep else f32s(reps)[b, s * n_rep:(s + 1) * n_rep, hh]
                    check_slot(c, b, hh, slot, f32s(At)[b, hh, s], f32s(Bc)[b, hh, s], R, fmt)
                    assert float(c.weight[b, hh, start + i]) == float(win[b, hh, i])
                for slot in set(range(n_cap)) - touched:
                    assert torch.equal(c.maps[b, hh, slot].view(torch.uint8), maps0[b, hh, slot])
                rest = [p for p in range(n_cap) if not start <= p < start + want]
                for p in rest:
                    assert float(c.weight[b, hh, p]) == (0.0 if reset else float(w0[b, hh, p]))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_append_live_chunk_resets_where_it_was_taken(fmt):
    note(f"append8 live {fmt}")
    h = hla()
    Bs, H, n_cap, dk, dv = 2, 2, 3, 128, 64
    c = make_cache(h, Bs, H, n_cap, dk, dv, 2, fmt, 61)
    c.count.copy_(torch.tensor([[0, 1], [2, 3]], dtype=torch.int32))
    randn, _ = rnd(62)
    A, S, reps = randn(Bs, H, dk, dk), randn(Bs, H, dk, dv), randn(Bs, 2, H, dk)
    A0, S0, m0 = A.clone(), S.clone(), c.maps.view(torch.uint8).clone()
    h.cache8_append(c, A, S, reps, reset_live=True)
    assert c.count.tolist() == [[1, 2], [3, 3]]
    for b in range(Bs):
        for hh in range(H):
            pos = 2 * b + hh
            if pos == 3:  # no room: nothing was appended, the live chunk goes on
                assert torch.equal(A[b, hh], A0[b, hh]) and torch.equal(S[b, hh], S0[b, hh])
                assert torch.equal(c.maps[b, hh].view(torch.uint8), m0[b, hh])
                continue
            check_slot(c, b, hh, int(c.order[b, hh, pos]), f32s(A0)[b, hh], f32s(S0)[b, hh], f32s(reps)[b, :, hh], fmt)
            assert torch.equal(A[b, hh], torch.eye(dk, device="cuda")) and not S[b, hh].any()
            assert float(c.weight[b, hh, pos]) == 0.0


# ------------------------------------------------------------------- weights and eviction
@pytest.mark.parametrize("B,H,N", [(1, 1, 1), (2, 3, 2), (1, 2, 64), (3, 2, 65), (2, 1, 127), (1, 2, 300)])
def test_gate_weights(B, H, N):
    note(f"gate weights {B} {H} {N}")
    _, rand = rnd(71)
    g = rand(B, H, N, N) ** 2
    g[rand(B, H, N, N) < 0.02] = float("nan")
    g[rand(B, H, N, N) < 0.02] = 2.5  # counts as 1
    up = torch.ones(N, N, dtype=torch.bool, device="cuda").triu()
    g.masked_fill_(up, float("inf"))  # never read
    n = torch.tensor([N, max(0, N - 3), 999][:B], dtype=torch.int32, device="cuda")
    for lens in (None, n):
        w = host(hla().gate_weights(g, tau=0.1, n_chunks=lens))
        for b in range(B):
            for hh in range(H):
                m = N if lens is None else min(int(lens[b]), N)
                want = o8.gate_weights(f32s(g)[b, hh], 0.1, m)
                assert np.max(np.abs(w[b, hh] - want)) <= N * EPS * max(1.0, want.max())  # N terms, summed in any order


def check_evict(w, count, budget, n_recent, order=None, in_place=False):
    h = hla()
    w0, c0 = f32s(w), count.cpu().numpy()
    Bs, H, n = w0.shape
    o0 = np.broadcast_to(np.arange(n), (Bs, H, n)) if order is None else order.cpu().numpy()
    out = (order, w, count) if in_place else None
    got = [t.cpu().numpy() for t in h.evict_chunks(w, count, budget, n_recent, order=order, out=out)]
    for b in range(Bs):
        for hh in range(H):
            ro, rw, rc = o8.evict(w0[b, hh], o0[b, hh], c0[b, hh], budget, n_recent)
            assert got[2][b, hh] == rc
            assert np.array_equal(got[0][b, hh], ro), f"order of row {b},{hh}"
            assert np.array_equal(got[1][b, hh], rw, equal_nan=True), f"weights of row {b},{hh}"


@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 200, 256, 1000, 1024, 1025, 2500, 4097])
def test_evict(n):
    note(f"evict n={n}")
    Bs, H = 2, 5
    _, rand = rnd(81)
    w = (rand(Bs, H, n) * 8).round() / 2  # many ties
    w[0, 0] = 1.0
    w[0, 1, ::3] = -0.0
    w[0, 1, 1::3] = 0.0
    w[1, 0] = rand(n) - 0.5
    w[1, 1, ::2] = float("inf")
    w[1, 2, ::2] = float("nan")
    w[1, 3] = -float("inf")
    order = rand(Bs, H, n).argsort(-1).to(torch.int32)
    count = torch.full((Bs, H), n, dtype=torch.int32, device="cuda")
    ragged = (rand(Bs, H) * (n + 1)).to(torch.int32)
    ragged[0, 0], ragged[1, 4] = n + 5, -2
    for budget, recent in {(n, 0), (n - 1, 0), (n // 2, n // 4), (n // 2, n // 2), (0, 0), (1, 1), (n + 7, 3)}:
        budget, recent = max(budget, 0), min(recent, max(budget, 0))
        for cnt in (count, ragged):
            check_evict(w, cnt, budget, recent, order)
            check_evict(w, cnt, budget, recent)
        check_evict(w.clone(), ragged.clone(), budget, recent, order.clone(), in_place=True)


def test_evict_widest():
    note("evict n=16384")
    _, rand = rnd(82)
    w = (rand(1, 2, 16384) * 64).round()
    w[0, 1, :8000] = 3.0
    count = torch.tensor([[16384, 16000]], dtype=torch.int32, device="cuda")
    check_evict(w, count, 1024, 8)
    check_evict(w, count, 15999, 8)


# ----------------------------------------------------------------------- as they are used
def serve(h, fmt, steps=5, C=64, T=300, n_cap=3, seed=91, gdn2=False, observe=None):
    """A prompt, its chunks cut to the cache's budget, decode steps with a live chunk that fills
    (the cache then drops its lightest chunk and takes it).  `observe` sees every step."""
    B, H, dk, dv, window = 1, 2, 64, 128, 16
    x = inputs.gen_tokens(B, T, H, dk, dv, dtype="bf16", seed=seed, alpha_mode="slow")
    q, k, v, beta, alpha = token_tensors(x)
    W = {n: torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).view(torch.bfloat16).cuda()
         for n, a in inputs.gen_pooler_weights(H, dk, dtype="bf16", seed=seed + 1).items()}
    r = h.hla_prefill(q, k, v, beta, alpha, pooler=W, window=window)
    c = h.cache8_alloc(B, H, n_cap, dk, dv, C // window, fmt)
    S, A = h.prefill_to_cache8(c, r, T)
    live = [k[:, T // C * C:].contiguous()]
    tail = T % C
    for s in range(steps):
        tok, gates, _, _ = token(B, H, dk, dv, "bf16", gdn2, seed + 10 + s)
        if observe:
            observe(c, tok, gates, S, A)
        else:
            h.gdn_decode8(*tok, *gates, S, A, c)
        live.append(tok[1].unsqueeze(1))
        tail += 1
        if tail == C:
            keys = torch.cat(live, 1).contiguous()
            reps = h.chunk_reps(keys, W, window=window).float()
            h.cache8_evict(c, n_cap - 1, 1)
            h.cache8_append(c, A, S, reps, reset_live=True)
            live, tail = [], 0
    return c, S, A


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_prompt_to_decode(fmt):
    """T = 300 leaves a live chunk of 44 tokens, which fills after 20 steps."""
    note(f"serve {fmt}")
    h = hla()
    c, S, A = serve(h, fmt, steps=24, observe=lambda c, tok, gates, S, A: check_decode(h, c, tok, gates, S, A))
    assert c.count.tolist() == [[3, 3]]
    assert torch.equal(c.order.sort(-1).values, torch.arange(3, dtype=torch.int32, device="cuda").expand(1, 2, 3))


def test_prompt_shorter_than_a_chunk_and_whole_chunks():
    h = hla()
    for T, held in ((40, 0), (64, 1), (128, 2)):
        note(f"serve T={T}")
        B, H, dk, dv = 2, 2, 128, 64
        x = inputs.gen_tokens(B, T, H, dk, dv, dtype="f32", seed=95, alpha_mode="slow")
        q, k, v, beta, alpha = token_tensors(x)
        r = h.hla_prefill(q, k, v, beta, alpha)
        c = make_cache(h, B, H, 4, dk, dv, 64, "int8", 96)
        c.count.fill_(4)
        S, A = h.prefill_to_cache8(c, r, T)
        assert c.count.unique().tolist() == [held]
        assert c.order.tolist() == [[[0, 1, 2, 3]] * H] * B
        if T == 40:
            assert torch.equal(A, r["At"][:, :, 0].float()) and torch.equal(S, r["Bc"][:, :, 0].float())
        else:
            assert torch.equal(A, torch.eye(dk, device="cuda").expand(B, H, dk, dk)) and not S.any()
        check_decode(h, c, *token(B, H, dk, dv, "f32", False, 97)[:2], S, A)


def test_step_in_a_graph_and_on_another_stream():
    """A decode step with eviction and append captured once and replayed, between eager work,
    against the same steps run eagerly; the eager run on a stream of its own."""
    note("cache8 graph")
    h = hla()
    Bs, H, n_cap, dk, dv = 2, 3, 200, 64, 64
    runs = []
    for mode in ("graph", "eager"):
        c = make_cache(h, Bs, H, n_cap, dk, dv, 2, "int8", 101)
        c.count.fill_(n_cap)
        tok, gates, S, A = token(Bs, H, dk, dv, "bf16", False, 102)
        randn, _ = rnd(103)
        reps = randn(Bs, 2, H, dk)
        o, gout = torch.empty(Bs, H, dv, device="cuda"), torch.empty(Bs, H, n_cap, device="cuda")
        ws = torch.empty(max(h.cache8_workspace_bytes(c), 16), dtype=torch.uint8, device="cuda")

        def step():
            h.gdn_decode8(*tok, *gates, S, A, c, o=o, gates_out=gout, ws=ws)
            h.cache8_evict(c, n_cap - 1, 1)
            h.cache8_append(c, A, S, reps, reset_live=True)

        side = torch.cuda.Stream()
        state = [t.clone() for t in (c.maps.view(torch.uint8), c.reps.view(torch.uint8), c.scale, c.order, c.count, c.weight, S, A)]
        live = (c.maps.view(torch.uint8), c.reps.view(torch.uint8), c.scale, c.order, c.count, c.weight, S, A)
        if mode == "graph":
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                step()
            for t, t0 in zip(live, state):
                t.copy_(t0)
        log = []
        for i in range(4):
            tok[0].copy_(token(Bs, H, dk, dv, "bf16", False, 110 + i)[0][0])
            if mode == "graph":
                g.replay()
            else:
                side.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(side):
                    step()
                torch.cuda.current_stream().wait_stream(side)
            torch.cuda.synchronize()
            log.append([t.clone() for t in (o, gout, *live)])
            (torch.ones(1000, device="cuda") * i).sum().item()
        runs.append(log)
    for a, b in zip(*runs):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_two_calls_on_one_cache_without_weights():
    """Two streams read one cache at once, each with its own live chunks and workspace."""
    note("cache8 two streams")
    h = hla()
    c = make_cache(h, 1, 4, 300, 128, 128, 2, "e4m3", 121, weights=False)
    c.count.fill_(300)
    toks = [token(1, 4, 128, 128, "bf16", False, 122 + i) for i in range(2)]
    alone = [h.gdn_decode8(*t, *g, S.clone(), A.clone(), c) for t, g, S, A in toks]
    streams = [torch.cuda.Stream() for _ in toks]
    torch.cuda.synchronize()
    outs = []
    for s, (t, g, S, A) in zip(streams, toks):
        with torch.cuda.stream(s):
            outs.append(h.gdn_decode8(*t, *g, S, A, c))
    torch.cuda.synchronize()
    for a, b in zip(alone, outs):
        assert torch.equal(a, b)


def test_refusals():
    note("cache8 refusals")
    h = hla()
    c = h.cache8_alloc(1, 2, 4, 64, 64, 2, "int8")
    with pytest.raises(AttributeError):
        c.count = c.count.clone()
    tok, gates, S, A = token(1, 2, 64, 64, "bf16", False, 131)
    bad = [dict(gates_in=torch.zeros(1, 2, 5, device="cuda")), dict(o=torch.zeros(1, 2, 64)), dict(tau=float("nan")),
           dict(gates_out=torch.zeros(1, 2, 4, device="cuda", dtype=torch.float64))]
    for kw in bad:
        with pytest.raises((ValueError, h.HlaError)):
            h.gdn_decode8(*tok, *gates, S, A, c, **kw)
    with pytest.raises(ValueError):
        h.gdn_decode8(tok[0][..., :32], *tok[1:], *gates, S, A, c)
    with pytest.raises(TypeError):
        h.gdn_decode8(*(t.half() for t in tok), *gates, S, A, c)
    with pytest.raises(ValueError):
        h.cache8_append(c, A, S)  # representatives missing
    with pytest.raises(ValueError):
        h.cache8_append(c, A, S, torch.zeros(1, 1, 2, 64, device="cuda"))
    with pytest.raises(h.HlaError):
        h.cache8_append(c, A, S, torch.zeros(1, 2, 2, 64, device="cuda"), src=torch.zeros(1, 2, 1, dtype=torch.int32, device="cuda"), reset_live=True)
    with pytest.raises(h.HlaError):
        h.evict_chunks(c.weight, c.count, 2, 3)
    with pytest.raises(h.HlaError):
        h.cache8_evict(c, -1)
    none = h.cache8_alloc(1, 2, 4, 64, 64, 0, "e4m3", weights=False)
    with pytest.raises(h.HlaError):
        h.gdn_decode8(*tok, *gates, S, A, none)  # nothing to score the chunks with
    with pytest.raises(ValueError):
        h.cache8_evict(none, 2)
    with pytest.raises(ValueError):
        h.Cache8(c.maps, c.reps, c.scale.cpu(), c.order, c.count)
    with pytest.raises(TypeError):
        h.Cache8(c.maps.float(), c.reps, c.scale, c.order, c.count)
    with pytest.raises(h.HlaError):
        h.cache8_alloc(1, 1, 1025, 64, 64)
