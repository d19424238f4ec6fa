"""Guard bands around everything the 8-bit chunk cache's calls are given: outputs, live matrices,
workspace and the cache's own arrays sit inside larger allocations whose bytes before and after hold
a canary pattern, which must still be there after the calls; outputs must be fully written."""
import pytest
import torch

import test_gpu_guards as guards
from gpu_util import note
from test_gpu_cache8 import hla, make_cache, rnd, token

pytestmark = pytest.mark.gpu


def guarded_copy(g, t):
    """t's contents in a guarded buffer of the same type (8-bit ones as bytes)."""
    raw = t.view(torch.uint8) if t.element_size() == 1 else t
    buf = g(tuple(t.shape), raw.dtype, output=False)
    buf.copy_(raw)
    return buf.view(t.dtype)


def guarded_cache(h, g, c):
    return h.Cache8(*(None if t is None else guarded_copy(g, t)
                      for t in (c.maps, c.reps, c.scale, c.order, c.count, c.weight)))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dk,dv,n_cap,n_rep,gdn2", [(128, 64, 11, 3, True), (64, 128, 200, 2, False), (128, 128, 130, 40, True),
                                                    (64, 64, 1, 1, False), (64, 64, 70, 0, True)], ids=str)
def test_decode_guards(fmt, dk, dv, n_cap, n_rep, gdn2):
    note(f"guards: cache8 decode {fmt} {dk} {dv} {n_cap} {n_rep}")
    h = hla()
    Bs, H = 1, 3
    g = guards.Guarded()
    c = guarded_cache(h, g, make_cache(h, Bs, H, n_cap, dk, dv, n_rep, fmt, 801))
    c.count.copy_(torch.tensor([[n_cap, n_cap // 2, 0]], dtype=torch.int32))
    held = [t.clone() for t in (c.maps.view(torch.uint8), c.scale, c.order, c.count)]
    tok, gates, S, A = token(Bs, H, dk, dv, "bf16", gdn2, 802)
    S, A = guarded_copy(g, S), guarded_copy(g, A)
    o, gout = g((Bs, H, dv), torch.float32), g((Bs, H, n_cap), torch.float32)
    ws = g((max(h.cache8_workspace_bytes(c), 16),), torch.uint8, output=False)
    gi = None if n_rep else 0.2 + 0.5 * rnd(803)[1](Bs, H, n_cap)
    step = h.gdn2_decode8 if gdn2 else h.gdn_decode8
    step(*tok, *gates, S, A, c, gates_in=gi, o=o, gates_out=gout, ws=ws)
    g.check(f"cache8 decode {fmt} n_cap={n_cap}")
    for t, t0 in zip((c.maps.view(torch.uint8), c.scale, c.order, c.count), held):
        assert torch.equal(t, t0)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype,dk,dv,n_rep", [("bf16", 128, 64, 3), ("f32", 64, 128, 1), ("f32", 128, 128, 17)], ids=str)
def test_append_and_evict_guards(fmt, dtype, dk, dv, n_rep):
    """A full cache after a reset, an append without room, an eviction in place, a live chunk."""
    note(f"guards: cache8 append and evict {fmt} {dtype} {dk} {dv}")
    h = hla()
    Bs, H, n_cap = 2, 3, 5
    randn, rand = rnd(811)
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    g = guards.Guarded()
    c = guarded_cache(h, g, h.cache8_alloc(Bs, H, n_cap, dk, dv, n_rep, fmt))
    At, Bc = (guarded_copy(g, randn(Bs, H, n_cap + 2, dk, w).to(dt)) for w in (dk, dv))
    reps = guarded_copy(g, randn(Bs, (n_cap + 2) * n_rep, H, dk).to(dt))
    h.cache8_append(c, At, Bc, reps, weight_in=rand(Bs, H, n_cap + 2), reset=True)
    h.cache8_append(c, At, Bc, reps)
    assert c.count.unique().tolist() == [n_cap]
    h.cache8_evict(c, n_cap - 1, 1)
    S, A = guarded_copy(g, randn(Bs, H, dk, dv)), guarded_copy(g, randn(Bs, H, dk, dk))
    live = guarded_copy(g, randn(Bs, n_rep, H, dk))
    h.cache8_append(c, A, S, live, reset_live=True)
    assert c.count.unique().tolist() == [n_cap] and not S.any()
    g.check(f"cache8 append {fmt} {dtype}")


@pytest.mark.parametrize("n", [1, 63, 200, 256, 700, 1024, 2000, 5000])
def test_weights_and_evict_guards(n):
    note(f"guards: gate weights and evict n={n}")
    h = hla()
    _, rand = rnd(821)
    g = guards.Guarded()
    if n <= 1024:
        h.gate_weights(guarded_copy(g, rand(2, 3, n, n)), tau=0.3, out=g((2, 3, n), torch.float32))
    out = (g((2, 3, n), torch.int32), g((2, 3, n), torch.float32), g((2, 3), torch.int32))
    count = guarded_copy(g, torch.full((2, 3), n, dtype=torch.int32, device="cuda"))
    h.evict_chunks(guarded_copy(g, rand(2, 3, n)), count, n // 2, n // 4, out=out)
    g.check(f"gate weights and evict n={n}")
