"""Extreme values in the split form of the 8-bit decode (few rows, a long cache), with enough
chunks held that segments are composed: large, tiny and zero maps, gates that are masked, not
finite or negative, slots that nothing names and slots out of range."""
import numpy as np
import pytest
import torch

from gpu_util import host, note
from test_cache8_bounds_cpu import SCALES
from test_gpu_cache8 import EPS, hla, make_cache, rnd, row_cache, token
from test_gpu_cache8_precision import check_close

pytestmark = pytest.mark.gpu
N_CAP = 130  # segments of 8 positions
SEG = 8


def split_cache(h, H, dk, dv, n_rep, fmt, seed):
    c = make_cache(h, 1, H, N_CAP, dk, dv, n_rep, fmt, seed)
    assert h.cache8_workspace_bytes(c) > 0
    return c


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("sa,used", SCALES, ids=str)
def test_scales_of_any_size_through_segments(fmt, sa, used):
    """A few chunks here and there, alone in their segments and together: maps that multiply |z| by a
    few hundred, maps near the identity, and the identity."""
    note(f"cache8 split scales {fmt} {sa}")
    h = hla()
    c = split_cache(h, 2, 64, 64, 0, fmt, 501)
    c.count.fill_(N_CAP)
    c.scale[..., 0] = sa
    gi = torch.zeros(1, 2, N_CAP, device="cuda")
    gi[..., used] = 0.75
    note(f"  worst {check_close(h, c, *token(1, 2, 64, 64, 'f32', False, 502), gates_in=gi, tau=0.5, seg=SEG):.3f}")


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("scored", [True, False])
def test_masks_and_unread_slots_through_segments(fmt, scored):
    """Counts about one segment's and the split's borders and out of range; the slots that no held
    position names hold NaN (0xFF in e4m3, NaN scales); gates NaN, infinite behind the last chunk,
    negative, and all below tau."""
    note(f"cache8 split masks {fmt} {scored}")
    h = hla()
    held = [63, 64, 65, 72, 73, 130, 500, -3]
    c = split_cache(h, len(held), 64, 128, 3, fmt, 511)
    c.count.copy_(torch.tensor([held], dtype=torch.int32))
    for hh, n in enumerate(held):
        n = min(max(n, 0), N_CAP)
        free = c.order[0, hh, n:].long()
        c.maps.view(torch.uint8)[0, hh, free] = 0xFF
        c.reps.view(torch.uint8)[0, hh, free] = 0xFF
        c.scale[0, hh, free] = float("nan")
    tok, gates, S, A = token(1, len(held), 64, 128, "f32", False, 512)
    if scored:
        check_close(h, c, tok, gates, S, A)
        check_close(h, c, tok, gates, S, A, tau=1.5)
        return
    _, rand = rnd(513)
    g = 0.1 * rand(1, len(held), N_CAP)
    g[0, 1, ::2] = float("nan")
    g[0, 2] = -0.05
    g[0, 3] = 0.0
    g[0, 5, ::3] = float("-inf")
    for hh, n in enumerate(held):
        g[0, hh, min(max(n, 0), N_CAP):] = float("inf")
    check_close(h, c, tok, gates, S, A, gates_in=g, tau=0.03)
    check_close(h, c, tok, gates, S, A, gates_in=g, tau=0.0)
    g[0, 5, ::3] = -0.02
    check_close(h, c, tok, gates, S, A, gates_in=g, tau=-float("inf"))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_slots_out_of_range_through_segments(fmt):
    note(f"cache8 split slots out of range {fmt}")
    h = hla()
    c = split_cache(h, 2, 64, 64, 2, fmt, 521)
    c.count.fill_(N_CAP)
    for p, s in ((2, 1 << 20), (50, -7), (51, N_CAP), (129, -(1 << 31))):
        c.order[0, :, p] = s
    want = c.order.clone()
    want[(want < 0) | (want >= N_CAP)] = N_CAP - 1
    outs = []
    for order in (c.order.clone(), want):
        c.order.copy_(order)
        tok, gates, S, A = token(1, 2, 64, 64, "bf16", False, 522)
        outs.append(h.gdn_decode8(*tok, *gates, S, A, c))
    assert torch.equal(*outs)


@pytest.mark.parametrize("n_cap", [20, 200])
@pytest.mark.parametrize("part", [0, 1], ids=["A", "B"])
def test_a_scale_that_is_not_finite_is_not_hidden(n_cap, part):
    """int8 has no stored byte that is not a number; a chunk's scale can be one."""
    note(f"cache8 scale not finite {n_cap} {part}")
    h = hla()
    for bad in (float("nan"), float("inf")):
        c = make_cache(h, 1, 3, n_cap, 64, 128, 0, "int8", 531)
        c.count.fill_(n_cap)
        tok, gates, S, A = token(1, 3, 64, 128, "f32", False, 532)
        gi = torch.full((1, 3, n_cap), 0.3, device="cuda")
        clean = host(h.gdn_decode8(*tok, *gates, S.clone(), A.clone(), c, gates_in=gi))
        c.scale[0, 1, int(c.order[0, 1, n_cap // 2 + 1]), part] = bad
        o = host(h.gdn_decode8(*tok, *gates, S.clone(), A.clone(), c, gates_in=gi))
        assert np.array_equal(o[0, [0, 2]], clean[0, [0, 2]])
        assert not np.isfinite(o[0, 1]).any()
        gi[0, 1, n_cap // 2 + 1] = 0.0  # and a skipped one is not read
        assert np.isfinite(host(h.gdn_decode8(*tok, *gates, S, A, c, gates_in=gi))).all()


@pytest.mark.parametrize("n_cap", [20, 200])
def test_e4m3_z_up_to_the_end_of_its_sums(n_cap):
    """The sums over e4m3 chunks are float32 sums of the stored numbers times z: z below 2^112 is
    exact, a larger one is right or not finite."""
    note(f"cache8 e4m3 largest z {n_cap}")
    h = hla()
    for zmax in (1.5 * 2.0 ** 111, 1.5 * 2.0 ** 127):
        c = make_cache(h, 1, 1, n_cap, 64, 64, 0, "e4m3", 541)
        c.count.fill_(n_cap)
        c.scale[..., 0] = 0.0  # A = I
        c.scale[..., 1] = 2.0 ** -20
        zero, one = torch.zeros(1, 1, 64, device="cuda"), torch.ones(1, 1, device="cuda")
        q = zero.clone()
        q[..., 3] = 1.0
        S, A = torch.zeros(1, 1, 64, 64, device="cuda"), torch.zeros(1, 1, 64, 64, device="cuda")
        A[0, 0, 3, 5] = zmax
        gi = torch.zeros(1, 1, n_cap, device="cuda")
        gi[..., n_cap // 2] = 1.0
        o = host(h.gdn_decode8(q, zero, zero, 0 * one, one, S, A, c, gates_in=gi, tau=0.5))[0, 0]
        ref = row_cache(c, 0, 0)[1][n_cap // 2][:, 5] * zmax
        right = np.abs(o - ref) <= 4 * EPS * np.abs(ref)
        assert np.all(right | ~np.isfinite(o))
        if zmax < 2.0 ** 112:
            assert np.all(right)
