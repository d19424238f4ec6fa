"""gdn_tree_decode in every form that sizes choose: one launch or two in front, a wave's gates of one chunk or of
several, one, two or four tiles of 16 nodes a workgroup, one or two chunks ahead, nodes in one group or in several.
A few rows, each repeated: every copy has the first one's bits, and the first ones are compared with the float64
recurrence (bounds: see test_gpu_tree)."""
import numpy as np
import pytest
import torch

from gated_deltanet_hybrid_amd import hla
from gpu_util import note
from test_gpu_tree import U, check, make, num, reference

pytestmark = pytest.mark.gpu

TOKENS = ("q", "k", "v", "beta", "alpha", "parent")


def forms(rows, n):
    """(tiles a workgroup, workgroups) of the chain kernel: the rule that these cases are meant to cover."""
    tiles, per = -(-n // 16), 1
    if tiles > 1 and rows * n > 16 * 256:
        per = 2
    if tiles > 2 and rows * ((tiles + 1) // 2) > 256:
        per = 4
    return per, rows * -(-tiles // per)


# (rows, n, dk, dv, dtype, n_cap, n_rep, tiles a workgroup, more than 256 workgroups)
CASES = [
    (300, 16, 128, 128, "bf16", 40, 3, 1, True),   # a serving batch; two chunks a wave's gates
    (300, 11, 128, 64, "f32", 9, 20, 1, True),
    (304, 1, 64, 64, "bf16", 6, 65, 1, True),
    (108, 33, 64, 128, "f32", 12, 3, 1, True),     # three groups of one tile
    (108, 33, 128, 128, "bf16", 5, 2, 1, True),
    (20, 40, 64, 128, "bf16", 7, 2, 1, False),     # two chunks ahead, three groups
    (40, 16, 128, 64, "f32", 7, 2, 1, False),
    (300, 17, 128, 128, "bf16", 5, 2, 2, True),
    (300, 32, 64, 128, "f32", 4, 3, 2, True),
    (100, 48, 128, 64, "bf16", 5, 17, 2, False),   # two groups, the second of one tile
    (100, 45, 128, 128, "f32", 3, 2, 2, False),
    (160, 50, 128, 128, "bf16", 4, 2, 4, False),
    (300, 64, 64, 128, "bf16", 3, 2, 4, True),
    (300, 40, 128, 64, "f32", 3, 2, 4, True),
    (1200, 64, 64, 64, "f32", 66, 2, 4, True),     # gates of eight and more chunks a wave
]


def repeated(x, times):
    d = {m: t.cuda() for m, t in x.items()}
    return {m: t.repeat(times, *[1] * (t.dim() - 1)).contiguous() for m, t in d.items()}


def answer(x, **kw):
    rest = {m: x[m] for m in ("At_cur", "At_cache", "Bc_cache", "reps_cache", "n_cache")}
    if "gates_in" in kw:
        rest["reps_cache"] = None
    return hla.gdn_tree_decode(*(x[m] for m in TOKENS), x["S_cur"], tau=0.3, **rest, **kw)


def against(o, x, ref, terms, what):
    """Within the bounds of magnitudes; and, where those have grown over many chunks, within as many roundings of the
    result's norm as there are terms (the maps here keep z's length)."""
    check(o, ref, terms, what)
    err = num(o.cpu()) - ref[0]
    assert np.linalg.norm(err) <= (6.0 * np.sqrt(terms / 3.0) + 24.0) * U * np.linalg.norm(ref[0]), what


@pytest.mark.parametrize("given", [False, True], ids=["scored", "given"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_forms(case, given):
    rows, n, dk, dv, dtype, n_cap, n_rep, per, many = case
    note(f"tree forms {case} {given}")
    assert forms(rows, n)[0] == per and (forms(rows, n)[1] > 256) == many
    H = 2
    x = make(2, n, H, dk, dv, dtype, n_cap, n_rep, seed=41)
    times = rows // (2 * H)
    assert times * 2 * H == rows
    big = repeated(x, times)
    terms = n + dk + n_cap * dk
    if given:  # a chunk is read by every third node of one tile alone, so other tiles skip it
        r = np.random.default_rng(43)
        g = np.where(r.random((2, n, H, n_cap)) < 0.4, 0.35 + 0.6 * r.random((2, n, H, n_cap)), 0.1)
        tiles = -(-n // 16)
        mine = np.arange(n)[:, None, None] // 16 == (np.arange(n_cap) % (tiles + 1))[None, None]
        g = torch.from_numpy(np.where(mine, g, 0.0).astype(np.float32))
        o = answer(big, gates_in=g.cuda().repeat(times, 1, 1, 1))
        ref = reference(x, 0.3, g)[0]
    else:
        gates = torch.full((2 * times, n, H, n_cap), 7.0, device="cuda")
        o = answer(big, gates_out=gates)
        ref, rg = reference(x, 0.3)
        assert not (np.abs(rg - 0.3) < 1e-5).any()
        assert torch.equal(gates, gates[:2].repeat(times, 1, 1, 1))
        smax = np.abs(num(x["reps_cache"])).max() * np.abs(num(x["q"])).max() * np.sqrt(dk)
        assert np.abs(num(gates[:2].cpu()) - rg).max() <= (6 * np.sqrt((dk + n_rep) / 3) + 24) * U * max(1.0, smax)
    assert torch.equal(o.view(torch.int32), o[:2].repeat(times, 1, 1, 1).view(torch.int32))
    against(o[:2], x, ref, terms, "o")
