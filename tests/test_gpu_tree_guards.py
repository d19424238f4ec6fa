"""Trees of drafted tokens: nothing is written outside the outputs and the workspace, what a call must not change
stays bit for bit, and calls on two streams with workspaces of their own do not meet."""
import numpy as np
import pytest
import torch

from gated_deltanet_hybrid_amd import hla
from gpu_util import note
from test_gpu_tree import make

pytestmark = pytest.mark.gpu

BAND = 4096
TOKENS = ("k", "v", "beta", "alpha", "parent")
LIVE = ("S_cur", "At_cur", "At_cache", "Bc_cache", "n_cache")


class Guarded:
    """Tensors between bands of one byte pattern."""

    def __init__(self):
        self.raws = []

    def empty(self, shape, dtype):
        size = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        raw = torch.full((size + 2 * BAND,), 0xA5, dtype=torch.uint8, device="cuda")
        self.raws.append(raw)
        return raw[BAND:BAND + size].view(dtype).view(*shape)

    def copy(self, t):
        out = self.empty(tuple(t.shape), t.dtype)
        out.copy_(t)
        return out

    def check(self):
        torch.cuda.synchronize()
        for raw in self.raws:
            assert (raw[:BAND] == 0xA5).all() and (raw[-BAND:] == 0xA5).all()


def on_device(x, times):
    return {m: t.cuda().repeat(times, *[1] * (t.dim() - 1)).contiguous() for m, t in x.items()}


# (Bs, copies, n, H, dk, dv, dtype, n_cap): one tile and several, one launch in front and two, few and many workgroups
CASES = [(1, 1, 1, 1, 64, 64, "f32", 1), (2, 1, 13, 2, 128, 128, "bf16", 5), (2, 1, 50, 1, 64, 128, "f32", 3),
         (2, 70, 17, 2, 128, 64, "bf16", 4), (2, 70, 64, 2, 64, 64, "f32", 3), (3, 30, 9, 3, 64, 128, "bf16", 7)]


@pytest.mark.parametrize("given", [False, True], ids=["scored", "given"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_decode_between_bands(case, given):
    Bs, times, n, H, dk, dv, dtype, n_cap = case
    note(f"tree guards {case} {given}")
    x = on_device(make(Bs, n, H, dk, dv, dtype, n_cap, 3, seed=61), times)
    B = Bs * times
    rest = {m: x[m] for m in ("At_cur", "At_cache", "Bc_cache", "n_cache")}
    gates = None if not given else torch.rand(B, n, H, n_cap, device="cuda")
    rest.update(dict(gates_in=gates) if given else dict(reps_cache=x["reps_cache"]))
    want_gates = torch.empty(B, n, H, n_cap, device="cuda")
    want = hla.gdn_tree_decode(x["q"], *(x[m] for m in TOKENS), x["S_cur"], tau=0.3, gates_out=want_gates, **rest)
    before = {m: t.clone() for m, t in x.items()}
    g = Guarded()
    o, out = g.empty((B, n, H, dv), torch.float32), g.empty((B, n, H, n_cap), torch.float32)
    ws = g.empty((hla.gdn_tree_workspace_bytes(B, H, n, dk, dv, n_cap),), torch.uint8)
    for fill in (0xA5, 0xFF):  # what the workspace held does not matter
        ws.fill_(fill)
        o.fill_(float("nan"))
        out.fill_(float("nan"))
        hla.gdn_tree_decode(x["q"], *(x[m] for m in TOKENS), x["S_cur"], tau=0.3, gates_out=out, o=o, ws=ws, **rest)
        g.check()
        assert torch.equal(o, want) and torch.equal(out, want_gates)
    assert all(torch.equal(x[m], before[m]) for m in x)


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_accept_between_bands(case):
    """Slots that no sequence appends to, sequences that accept nothing, and the bands stay as they were."""
    Bs, times, n, H, dk, dv, dtype, n_cap = case
    note(f"accept guards {case}")
    x = on_device(make(Bs, n, H, dk, dv, dtype, n_cap, 1, seed=62), times)
    B = Bs * times
    r = np.random.default_rng(63)
    count = r.integers(0, n_cap + 1, B).astype(np.int32)
    commit, node = r.integers(0, 2, B).astype(np.int32), r.integers(-1, n, B).astype(np.int32)
    count[0], commit[0] = n_cap, 1  # full: left as it is
    x["n_cache"] = torch.from_numpy(count).cuda()
    g = Guarded()
    live = {m: g.copy(x[m]) for m in LIVE}
    parent = x["parent"].cpu().numpy()
    hla.gdn_tree_accept(*(x[m] for m in TOKENS), torch.from_numpy(node).cuda(), commit=torch.from_numpy(commit).cuda(), **live)
    g.check()
    for b in range(B):
        appended = bool(commit[b]) and count[b] < n_cap
        assert int(live["n_cache"][b]) == count[b] + appended
        for m in ("At_cache", "Bc_cache"):
            others = [j for j in range(n_cap) if not (appended and j == count[b])]
            assert torch.equal(live[m][b][:, others], x[m][b][:, others])
        if not appended and (node[b] < 0 or parent[b, node[b]] < -1):
            assert torch.equal(live["S_cur"][b], x["S_cur"][b]) and torch.equal(live["At_cur"][b], x["At_cur"][b])
        if appended:
            eye = torch.eye(dk, device="cuda").expand(H, dk, dk)
            assert (live["S_cur"][b] == 0).all() and torch.equal(live["At_cur"][b], eye)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_two_streams_at_once(dtype):
    note(f"tree two streams {dtype}")
    shapes = [(2, 20, 2, 128, 64, dtype, 9, 5), (3, 60, 2, 64, 128, dtype, 6, 2)]
    xs = [{m: t.cuda() for m, t in make(*s, seed=64 + i).items()} for i, s in enumerate(shapes)]

    def call(x):
        return hla.gdn_tree_decode(x["q"], *(x[m] for m in TOKENS), x["S_cur"], tau=0.3, reps_cache=x["reps_cache"],
                                   **{m: x[m] for m in LIVE if m != "S_cur"})

    want = [call(x) for x in xs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in xs], [[], []]
    for _ in range(6):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(call(xs[i]))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(w, o) for o in g)
