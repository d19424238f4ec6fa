"""What prefill_to_cache8 refuses, on the host: each refusal comes before any library call, so a
prefill's result and a cache of the right shapes are enough (no GPU needed)."""
import types

import pytest
import torch

from gated_deltanet_hybrid_amd import hla


def result(T, C=64, n_rep=None, S0=None, dk=64, dv=64):
    N = -(-T // C)
    n_rep = C if n_rep is None else n_rep
    z = torch.zeros
    return dict(At=z(1, 2, N, dk, dk), Bc=z(1, 2, N, dk, dv), gates=z(1, 2, N, N), o=z(1, T, 2, dv),
                reps=z(1, T if n_rep == C else N * n_rep, 2, dk), n_rep=n_rep, C=C, S0=S0, tau=1e-3)


def cache(n_rep):
    return types.SimpleNamespace(Bs=1, H=2, n_cap=4, n_rep=n_rep, dk=64, dv=64)


@pytest.fixture(autouse=True)
def nothing_is_enqueued(monkeypatch):
    class Enqueued(Exception):
        pass

    def call(*a):
        raise Enqueued
    monkeypatch.setattr(hla, "_call", call)
    # (host tensors: what is not refused ends at the first device tensor it asks for, or here)
    return Enqueued


def test_representatives_of_another_size_are_refused():
    # 96 tokens are two chunks: as many keys as two chunks of 48 representatives would have rows
    with pytest.raises(ValueError, match="representatives"):
        hla.prefill_to_cache8(cache(48), result(96), 96)
    for held in (2, 32, 128):
        with pytest.raises(ValueError, match="representatives"):
            hla.prefill_to_cache8(cache(held), result(200), 200)
        with pytest.raises(ValueError, match="representatives"):
            hla.prefill_to_cache8(cache(held), result(200, n_rep=4), 200)


@pytest.mark.parametrize("T,C", [(127, 64), (65, 64), (96, 48), (96, 128), (192, 64), (0, 64)])
def test_another_length_or_chunk_is_refused(T, C):
    with pytest.raises(ValueError, match="T and C"):
        hla.prefill_to_cache8(cache(64), result(96), T, C=C)


def test_a_single_chunk_of_another_size_is_refused():
    """64 tokens are one whole chunk of 64, and one unfinished chunk of 128."""
    with pytest.raises(ValueError, match="T and C"):
        hla.prefill_to_cache8(cache(0), result(64, C=128), 64)


def test_an_initial_state_is_refused():
    with pytest.raises(ValueError, match="S0"):
        hla.prefill_to_cache8(cache(64), result(96, S0=torch.zeros(1, 2, 64, 64)), 96)
