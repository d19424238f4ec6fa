"""Calls on the 8-bit chunk cache with tensors as a program holds them: views that begin where only
4-byte alignment is left, representatives in a window of a longer row, numbers of representatives on
both sides of a block of scores, long rows evicted in place in a graph, a prompt on another stream."""
import numpy as np
import pytest
import torch

import oracle.cache8 as o8
from gpu_util import host, note
from test_gpu_cache8 import EPS, check_slot, f32s, hla, make_cache, rnd, token
from test_gpu_cache8_precision import check_close
from test_gpu_cache8_prompt import prompt

pytestmark = pytest.mark.gpu


def offset(t, n):
    """t's contents n elements into an allocation of its own."""
    buf = torch.empty(t.numel() + n, dtype=t.dtype, device=t.device)
    view = buf[n:].view(t.shape)
    view.copy_(t)
    return view


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("n_cap,n_rep", [(70, 3), (12, 5)])
@pytest.mark.parametrize("gdn2", [False, True])
def test_decode_of_offset_views(fmt, n_cap, n_rep, gdn2):
    """Tokens, gates and outputs 4 bytes into their allocations: the same bits as from their starts."""
    note(f"cache8 offset views {fmt} {n_cap} {gdn2}")
    h = hla()
    step = h.gdn2_decode8 if gdn2 else h.gdn_decode8
    outs = []
    for off in (0, 1):
        c = make_cache(h, 1, 3, n_cap, 64, 128, n_rep, fmt, 901)
        c.count.fill_(n_cap)
        tok, gates, S, A = token(1, 3, 64, 128, "bf16", gdn2, 902)
        tok, gates = [offset(t, 2 * off) for t in tok], [offset(t, off) for t in gates]
        o, gout = (offset(torch.full(s, float("nan"), device="cuda"), off) for s in ((1, 3, 128), (1, 3, n_cap)))
        step(*tok, *gates, S, A, c, o=o, gates_out=gout)
        gi = offset(0.5 * gout + 0.1, off)
        o2 = step(*tok, *gates, S, A, c, gates_in=gi)
        outs.append([t.clone() for t in (o, gout, o2, S, A, c.weight)])
    for a, b in zip(*outs):
        assert torch.equal(a, b)


@pytest.mark.parametrize("N", [64, 100, 256])
def test_gate_weights_of_an_offset_matrix(N):
    """A matrix whose rows are not 16-byte aligned takes the loads of single numbers."""
    note(f"gate weights of an offset matrix {N}")
    g = offset(rnd(911)[1](2, 3, N, N), 1)
    w = host(hla().gate_weights(g, tau=0.2))
    for b in range(2):
        for hh in range(3):
            want = o8.gate_weights(f32s(g)[b, hh], 0.2, N)
            assert np.max(np.abs(w[b, hh] - want)) <= N * EPS * max(1.0, want.max())


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_representatives_in_a_window(fmt, dtype):
    """Rows of a longer allocation ([B, ld, H, dk], a token window), more of them than are read."""
    note(f"append8 representatives in a window {fmt} {dtype}")
    h = hla()
    randn, _ = rnd(921)
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    B, H, n, n_rep, dk, dv = 3, 2, 4, 5, 64, 64
    c = h.cache8_alloc(B, H, 6, dk, dv, n_rep, fmt)
    At, Bc = randn(B, H, n, dk, dk).to(dt), randn(B, H, n, dk, dv).to(dt)
    reps = randn(B, 50, H, dk).to(dt)[:, 7:7 + n * n_rep + 3]
    h.cache8_append(c, At, Bc, reps)
    for b in range(B):
        for hh in range(H):
            for i in range(n):
                check_slot(c, b, hh, i, f32s(At)[b, hh, i], f32s(Bc)[b, hh, i], f32s(reps)[b, i * n_rep:(i + 1) * n_rep, hh], fmt)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("n_rep", [7, 16, 31, 32, 33, 64, 127, 255])
@pytest.mark.parametrize("n_cap,dk", [(37, 64), (70, 128)])
def test_numbers_of_representatives(fmt, n_rep, n_cap, dk):
    note(f"cache8 representatives {fmt} {n_rep} {n_cap}")
    h = hla()
    c = make_cache(h, 1, 2, n_cap, dk, 64, n_rep, fmt, 931)
    c.count.copy_(torch.tensor([[n_cap, n_cap - 3]], dtype=torch.int32))
    check_close(h, c, *token(1, 2, dk, 64, "f32", False, 932))


@pytest.mark.parametrize("n", [300, 1024, 2500, 9000])
def test_long_rows_evicted_in_place_in_a_graph(n):
    """Captured once and replayed on new weights, between eager work: each replay as the oracle says."""
    note(f"evict in a graph n={n}")
    h = hla()
    _, rand = rnd(941)
    w, order, count = torch.empty(1, 3, n, device="cuda"), torch.empty(1, 3, n, dtype=torch.int32, device="cuda"), \
        torch.empty(1, 3, dtype=torch.int32, device="cuda")

    def fill(i):
        w.copy_((rand(1, 3, n) * (20 + i)).round())
        order.copy_(rand(1, 3, n).argsort(-1).to(torch.int32))
        count.copy_(torch.tensor([[n, n - 7, n // 2]], dtype=torch.int32))

    fill(0)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        h.evict_chunks(w, count, n // 2, n // 8, order=order, out=(order, w, count))
    for i in range(4):
        fill(i)
        before = [t.cpu().numpy().copy() for t in (w, order, count)]
        g.replay()
        torch.cuda.synchronize()
        for hh in range(3):
            ro, rw, rc = o8.evict(before[0][0, hh], before[1][0, hh], before[2][0, hh], n // 2, n // 8)
            assert np.array_equal(order[0, hh].cpu().numpy(), ro) and np.array_equal(w[0, hh].cpu().numpy(), rw)
            assert int(count[0, hh]) == rc
        (torch.ones(1000, device="cuda") * i).sum().item()


def test_evict_without_an_order_in_place():
    """The weights and the count in place, the order new."""
    note("evict without an order, in place")
    _, rand = rnd(951)
    for n in (60, 700):
        w, count = rand(2, 2, n), torch.full((2, 2), n, dtype=torch.int32, device="cuda")
        w0, order = f32s(w), torch.empty(2, 2, n, dtype=torch.int32, device="cuda")
        hla().evict_chunks(w, count, n // 3, 2, out=(order, w, count))
        for b in range(2):
            for hh in range(2):
                ro, rw, rc = o8.evict(w0[b, hh], np.arange(n), n, n // 3, 2)
                assert np.array_equal(order[b, hh].cpu().numpy(), ro) and np.array_equal(f32s(w)[b, hh], rw)
                assert int(count[b, hh]) == rc


@pytest.mark.parametrize("budget", [None, 3, 0])
def test_a_prompt_on_another_stream(budget):
    """The whole way from the prompt to a step on a stream of its own, as on the default one."""
    note(f"cache8 prompt on another stream, budget {budget}")
    h = hla()
    k, r = prompt(h, 2, 500, 2, 64, 64)
    torch.cuda.synchronize()
    outs = []
    for stream in (torch.cuda.current_stream(), torch.cuda.Stream()):
        with torch.cuda.stream(stream):
            c = h.cache8_alloc(2, 2, 6, 64, 64, 64, "int8")
            S, A = h.prefill_to_cache8(c, r, 500, budget=budget)
            tok, gates, _, _ = token(2, 2, 64, 64, "f32", False, 961)
            o = h.gdn_decode8(*tok, *gates, S, A, c)
        torch.cuda.synchronize()
        outs.append([t.clone() for t in (o, S, A, c.maps.view(torch.uint8), c.order, c.count, c.weight)])
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    assert c.count.unique().tolist() == [6 if budget is None else budget]


@pytest.mark.parametrize("dk,n_cap", [(64, 20), (128, 20), (64, 130)])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_chunks_that_clear_the_state(fmt, dk, n_cap):
    """Maps with A = 0 (a strong decay) read with gates up to 1: z all but vanishes at every chunk, and
    what is left is as close as float32's own subtraction leaves it."""
    note(f"cache8 clearing chunks {fmt} {dk} {n_cap}")
    h = hla()
    c = h.cache8_alloc(1, 2, n_cap, dk, 64, 0, fmt)
    randn, rand = rnd(971)
    h.cache8_append(c, torch.zeros(1, 2, n_cap, dk, dk, device="cuda"), randn(1, 2, n_cap, dk, 64))
    gi = 1.0 - 0.9 * rand(1, 2, n_cap) ** 4
    check_close(h, c, *token(1, 2, dk, 64, "f32", False, 972), gates_in=gi, seg=8 if n_cap > 64 else None)
