"""Appending chunks whose numbers are extreme: a block that holds a NaN or an infinity is stored so
that every decode that reads it shows it; blocks at the end of float32's range are stored exactly."""
import numpy as np
import pytest
import torch

from gpu_util import host, note
from test_gpu_cache8 import TORCH, check_slot, f32s, hla, make_cache, rnd, token, values

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


def chunks(Bs, H, L, dk, dv, n_rep, dtype, seed):
    randn, _ = rnd(seed)
    At = (torch.eye(dk, device="cuda") + randn(Bs, H, L, dk, dk) * 0.1).to(TORCH[dtype])
    return At, randn(Bs, H, L, dk, dv).to(TORCH[dtype]), randn(Bs, L * n_rep, H, dk).to(TORCH[dtype])


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype,dk,dv,n_rep", [("bf16", 128, 128, 3), ("f32", 64, 128, 2), ("f32", 128, 64, 17)], ids=str)
def test_blocks_that_are_not_finite(fmt, dtype, dk, dv, n_rep):
    """Each of A - I, B and the representatives with one bad number, at the first and the last place and
    between, or with nothing else: scale NaN, stored zeros, and the chunk's other blocks as ever."""
    note(f"append8 not finite {fmt} {dtype} {dk} {dv}")
    h = hla()
    L = 15
    At, Bc, reps = chunks(1, 2, L, dk, dv, n_rep, dtype, 701)
    c = h.cache8_alloc(1, 2, L, dk, dv, n_rep, fmt)
    bad = {}
    for i in range(12):
        part, value = i % 3, (NAN, INF, -INF, NAN)[i // 3]
        block = (At[0, 0, i], Bc[0, 0, i], reps[0, i * n_rep:(i + 1) * n_rep, 0])[part]
        if i >= 9:
            block.fill_(value)
        else:
            r, col = ((0, 0), (block.shape[0] // 2, 17), (block.shape[0] - 1, block.shape[1] - 1))[i // 3]
            block[r, col] = value
        bad[i] = part
    h.cache8_append(c, At, Bc, reps)
    torch.cuda.synchronize()
    assert c.count.tolist() == [[L, L]]
    for hh in range(2):
        for i in range(L):
            if hh or i not in bad:
                check_slot(c, 0, hh, i, f32s(At)[0, hh, i], f32s(Bc)[0, hh, i],
                           f32s(reps)[0, i * n_rep:(i + 1) * n_rep, hh], fmt)
                continue
            part = bad[i]
            assert np.isnan(c.scale[0, 0, i].tolist()).tolist() == [part == x for x in range(3)] + [False]
            m = values(c.maps[0, 0, i].view(torch.uint8).view(c.maps.dtype))
            stored = (m[:dk], m[dk:], values(c.reps[0, 0, i]))
            assert not stored[part].any()
            assert all(stored[x].any() for x in range(3) if x != part)


@pytest.mark.parametrize("n_cap", [6, 200])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_decode_shows_what_was_not_finite(n_cap, fmt, dtype):
    """Rows whose chunk held a NaN in A, in B or in its keys; the row without one is as ever.  A chunk
    without a gate (its keys were NaN) is not read, as a NaN gate is below every threshold."""
    note(f"append8 then decode, not finite {n_cap} {fmt} {dtype}")
    h = hla()
    dk, dv, n_rep, at = 64, 64, 2, n_cap // 2
    At, Bc, reps = chunks(1, 4, n_cap, dk, dv, n_rep, dtype, 711)
    At = (torch.eye(dk, device="cuda") + (At.float() - torch.eye(dk, device="cuda")) * 0.02).to(TORCH[dtype])
    caches = [h.cache8_alloc(1, 4, n_cap, dk, dv, n_rep, fmt) for _ in range(2)]
    h.cache8_append(caches[0], At, Bc, reps)
    At[0, 0, at, 5, 6] = NAN
    Bc[0, 1, at, 0, 0] = -INF
    reps[0, at * n_rep + 1, 2, 63] = NAN
    h.cache8_append(caches[1], At, Bc, reps)
    tok, gates, S, A = token(1, 4, dk, dv, dtype, False, 712)
    outs, gouts = [], []
    for c in caches:
        gout = torch.empty(1, 4, n_cap, device="cuda")
        outs.append(host(h.gdn_decode8(*tok, *gates, S.clone(), A.clone(), c, gates_out=gout)))
        gouts.append(host(gout))
    clean, o = outs
    assert np.isfinite(clean).all()
    assert np.isnan(o[0, :2]).all()
    assert np.isfinite(o[0, 2]).all() and np.isnan(gouts[1][0, 2, at]) and np.isnan(gouts[1]).sum() == 1
    assert float(caches[1].weight[0, 2, at]) == 0.0
    assert np.array_equal(o[0, 3], clean[0, 3])


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_a_live_chunk_that_is_not_finite_stays_so(fmt):
    """A NaN in the live state shows in every decode; once the chunk is in the cache it still does."""
    note(f"append8 live chunk not finite {fmt}")
    h = hla()
    c = make_cache(h, 1, 2, 4, 64, 64, 0, fmt, 721)
    c.count.fill_(2)
    tok, gates, S, A = token(1, 2, 64, 64, "f32", False, 722)
    S[0, 0, 3, 7] = NAN
    gi = torch.full((1, 2, 4), 0.5, device="cuda")
    for _ in range(2):
        o = host(h.gdn_decode8(*tok, *gates, S, A, c, gates_in=gi))
        assert np.isnan(o[0, 0]).any() and np.isfinite(o[0, 1]).all()
        h.cache8_append(c, A, S, reset_live=True)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("exponent", [127, 126, 100, -99, -100, -101, -130])
def test_blocks_at_the_ends_of_the_range(fmt, exponent):
    """Largest magnitudes up to float32's end (whose reciprocal is below its smallest normal number)
    and about the one below which zeros are stored."""
    note(f"append8 magnitude 2^{exponent} {fmt}")
    h = hla()
    randn, rand = rnd(731)
    m = 2.0 ** exponent
    B = (rand(1, 1, 1, 64, 64) * 2 - 1) * m
    B[0, 0, 0, 9, 9] = 1.5 * m
    A = torch.eye(64, device="cuda").view(1, 1, 1, 64, 64).clone()
    R = (rand(1, 2, 1, 64) * 2 - 1) * m
    c = h.cache8_alloc(1, 1, 1, 64, 64, 2, fmt)
    h.cache8_append(c, A, B, R)
    check_slot(c, 0, 0, 0, f32s(A)[0, 0, 0], f32s(B)[0, 0, 0], f32s(R)[0, :, 0], fmt)
