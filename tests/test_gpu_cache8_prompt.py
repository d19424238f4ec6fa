"""From a prompt to the 8-bit chunk cache on the GPU: both recurrences, what the call returns and
leaves alone, the units of the weights it hands to the decode steps, and the prefills it refuses."""
import numpy as np
import pytest
import torch

import oracle.cache8 as o8
from gated_deltanet_hybrid_amd import inputs
from gpu_util import f32, note, token_tensors
from test_gpu_cache8 import EPS, check_decode, check_slot, f32s, hla, token

pytestmark = pytest.mark.gpu
C = 64


def prompt(h, B, T, H, dk, dv, dtype="f32", gdn2=False, seed=301, chunk=C, **kw):
    x = inputs.gen_tokens(B, T, H, dk, dv, dtype=dtype, seed=seed, alpha_mode="slow")
    q, k, v, beta, alpha = token_tensors(x)
    if not gdn2:
        return k, h.hla_prefill(q, k, v, beta, alpha, C=chunk, **kw)
    g = inputs.gen_gdn2_gates(B, T, H, dk, dv, seed=seed, alpha_mode="slow")
    return k, h.gdn2_hla_prefill(q, k, v, *(f32(g[n]) for n in ("a", "b", "w")), C=chunk, **kw)


def check_cache(c, r, k, n, chunk=C):
    """Every held position's stored values are those of the source chunk `kept[p]`."""
    for b in range(c.Bs):
        for hh in range(c.H):
            for p, src in enumerate(n[b][hh]):
                slot = int(c.order[b, hh, p])
                reps = None if not c.n_rep else f32s(k)[b, src * chunk:(src + 1) * chunk, hh]
                check_slot(c, b, hh, slot, f32s(r["At"])[b, hh, src], f32s(r["Bc"])[b, hh, src], reps,
                           "int8" if c.maps.dtype == torch.int8 else "e4m3")


@pytest.mark.parametrize("fmt,dtype,dk,dv,n_rep", [("int8", "bf16", 128, 64, C), ("e4m3", "f32", 64, 128, C),
                                                   ("int8", "f32", 64, 64, 0)], ids=str)
def test_gdn2_prompt_to_decode(fmt, dtype, dk, dv, n_rep):
    """Gated DeltaNet-2: 200 tokens leave three chunks and a live one of 8; scored by the chunks'
    own keys, or by the caller's gates over a cache that holds none."""
    note(f"cache8 gdn2 prompt {fmt} {dtype} {dk} {dv} {n_rep}")
    h = hla()
    B, H, T = 2, 2, 200
    k, r = prompt(h, B, T, H, dk, dv, dtype, gdn2=True)
    c = h.cache8_alloc(B, H, 5, dk, dv, n_rep, fmt)
    S, A = h.prefill_to_cache8(c, r, T)
    assert c.count.tolist() == [[3, 3]] * B
    check_cache(c, r, k, [[[0, 1, 2]] * H] * B)
    assert torch.equal(A, r["At"][:, :, 3].float()) and torch.equal(S, r["Bc"][:, :, 3].float())
    for s in range(3):
        tok, gates, _, _ = token(B, H, dk, dv, dtype, True, 310 + s)
        gi = None if n_rep else torch.full((B, H, 5), 0.25, device="cuda")
        check_decode(h, c, tok, gates, S, A, gates_in=gi)


@pytest.mark.parametrize("T", [40, 150])
def test_the_live_chunk_is_not_the_prefills(T):
    """One row: the last chunk's maps are contiguous as they lie in the prefill's tensors.  A decode
    step, which updates the live chunk in place, leaves the prefill's result as it was."""
    note(f"cache8 live chunk of its own T={T}")
    h = hla()
    k, r = prompt(h, 1, T, 1, 64, 64)
    At, Bc = r["At"].clone(), r["Bc"].clone()
    c = h.cache8_alloc(1, 1, 4, 64, 64, C, "int8")
    S, A = h.prefill_to_cache8(c, r, T)
    tok, gates, _, _ = token(1, 1, 64, 64, "f32", False, 321)
    h.gdn_decode8(*tok, *gates, S, A, c)
    assert torch.equal(r["At"], At) and torch.equal(r["Bc"], Bc)
    S2, A2 = h.prefill_to_cache8(c, r, T)  # and the same prompt enters again
    assert torch.equal(A2, At[:, :, -1]) and torch.equal(S2, Bc[:, :, -1])


@pytest.mark.parametrize("tau", [1e-3, 0.4, 0.5, 2.0])
def test_weights_are_of_the_gates_that_the_prefill_kept(tau):
    """Without a tau of its own the call weighs by the prefill's: chunks that it skipped weigh nothing."""
    note(f"cache8 weights by the prefill's tau={tau}")
    h = hla()
    k, r = prompt(h, 1, 300, 2, 64, 64, tau=tau)
    weights = []
    for kw in ({}, dict(tau=tau)):
        c = h.cache8_alloc(1, 2, 6, 64, 64, 0, "int8")
        h.prefill_to_cache8(c, r, 300, **kw)
        weights.append(c.weight)
        for hh in range(2):
            kept = o8.gate_weights(f32s(r["gates"])[0, hh], tau, 5)[:4]
            assert np.array_equal(c.weight[0, hh, :4].cpu().numpy() > 0, kept > 0)
    assert torch.equal(*weights)


@pytest.mark.parametrize("chunk", [64, 128])
@pytest.mark.parametrize("tau", [1e-3, 0.4])
def test_weights_count_tokens(chunk, tau):
    """A prompt's gate is one query chunk's, a decode step's one token's: the prompt's weights count
    each gate once for every token of a chunk, of the gates that the prefill itself kept."""
    note(f"cache8 weights by token C={chunk} tau={tau}")
    h = hla()
    B, H, T = 1, 2, 5 * chunk + 10
    k, r = prompt(h, B, T, H, 128, 64, "bf16", chunk=chunk, tau=tau)
    for gate_tokens in (None, 1):
        c = h.cache8_alloc(B, H, 8, 128, 64, 0, "e4m3")
        S, A = h.prefill_to_cache8(c, r, T, C=chunk, **({} if gate_tokens is None else dict(gate_tokens=gate_tokens)))
        for hh in range(H):
            want = o8.gate_weights(f32s(r["gates"])[0, hh], tau, 6)[:5] * (chunk if gate_tokens is None else 1)
            got = c.weight[0, hh].tolist()
            assert np.all(np.abs(np.array(got[:5]) - want) <= 8 * EPS * max(1.0, want.max()))
            assert got[5:] == [0.0] * 3
    gi = torch.full((B, H, 8), 0.5, device="cuda")
    before = c.weight.clone()
    tok, gates, _, _ = token(B, H, 128, 64, "bf16", False, 331)
    h.gdn_decode8(*tok, *gates, S, A, c, gates_in=gi)
    assert torch.equal(c.weight[..., :5], before[..., :5] + 0.5)  # one token's gate


def test_prefills_that_do_not_fit_are_refused():
    """The same refusals as on the host, of results that a prefill gave."""
    note("cache8 prompt refusals")
    h = hla()
    k, r = prompt(h, 1, 96, 2, 64, 64)
    assert r["reps"].shape[1] == 2 * 48
    with pytest.raises(ValueError):
        h.prefill_to_cache8(h.cache8_alloc(1, 2, 4, 64, 64, 48, "int8"), r, 96)
    c = h.cache8_alloc(1, 2, 4, 64, 64, C, "int8")
    for T, chunk in ((127, 64), (65, 64), (96, 48)):
        with pytest.raises(ValueError):
            h.prefill_to_cache8(c, r, T, C=chunk)
    _, r0 = prompt(h, 1, 96, 2, 64, 64, S0=torch.ones(1, 2, 64, 64, device="cuda"))
    _, r2 = prompt(h, 1, 96, 2, 64, 64, gdn2=True, S0=torch.ones(1, 2, 64, 64, device="cuda"))
    for bad in (r0, r2):
        with pytest.raises(ValueError, match="S0"):
            h.prefill_to_cache8(c, bad, 96)
    assert not c.count.any()
    h.prefill_to_cache8(c, r, 96)
    assert c.count.tolist() == [[1, 1]]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_gdn2_live_chunk_enters_the_cache(fmt):
    """Gated DeltaNet-2 as it is served: 250 tokens, then steps until the live chunk is complete, the full
    cache drops its lightest chunk and takes it, and steps over the new set."""
    note(f"cache8 gdn2 serve {fmt}")
    h = hla()
    B, H, T, dk, dv = 1, 2, 250, 64, 128
    k, r = prompt(h, B, T, H, dk, dv, "bf16", gdn2=True)
    c = h.cache8_alloc(B, H, 3, dk, dv, C, fmt)
    S, A = h.prefill_to_cache8(c, r, T)
    live = [k[:, T // C * C:]]
    for s in range(9):
        tok, gates, _, _ = token(B, H, dk, dv, "bf16", True, 350 + s)
        check_decode(h, c, tok, gates, S, A)
        live.append(tok[1].unsqueeze(1))
        if (T + s + 1) % C == 0:
            keys, S0, A0 = torch.cat(live, 1).float().contiguous(), f32s(S), f32s(A)
            assert keys.shape[1] == C
            weights = c.weight.clone()
            h.cache8_evict(c, 2, 1)
            h.cache8_append(c, A, S, keys, reset_live=True)
            for hh in range(H):
                assert c.weight[0, hh, 2] == 0 and c.weight[0, hh, 1] == weights[0, hh, 2]  # the newest stayed
                check_slot(c, 0, hh, int(c.order[0, hh, 2]), A0[0, hh], S0[0, hh], f32s(keys)[0, :, hh], fmt)
    assert c.count.tolist() == [[3, 3]] and s > 6
