"""Trees of drafted tokens without a cache, host side: a call that could not fill gates_out is refused, and so are
live matrices without the cache they are read with."""
import pytest
import torch

from gated_deltanet_hybrid_amd import hla
from test_abi_la_tree_cpu import HIP, NULL_ARG, TREE, tree_tensors

AT_CUR, GATES_OUT = 13, 23  # places in TREE


def test_gates_out_needs_the_cache():
    lib = hla.library()
    a = list(TREE)
    a[AT_CUR] = None
    assert lib.hla_gdn_tree_decode(*a) == NULL_ARG
    a[GATES_OUT] = None
    a[3] = 96  # refused for its width before anything is enqueued: without gates_out the call is sound so far
    assert lib.hla_gdn_tree_decode(*a) not in (NULL_ARG, HIP)


def test_the_binding_refuses_gates_out_without_the_cache():
    t, q = tree_tensors(), torch.zeros(2, 5, 3, 64)
    with pytest.raises(ValueError, match="gates_out"):
        hla.gdn_tree_decode(q, **t, gates_out=torch.zeros(2, 5, 3, 4))


@pytest.mark.parametrize("missing", ["At_cache", "Bc_cache", "n_cache"])
def test_the_binding_refuses_live_matrices_without_their_cache(missing):
    t, q = tree_tensors(), torch.zeros(2, 5, 3, 64)
    cache = dict(At_cur=torch.zeros(2, 3, 64, 64), At_cache=torch.zeros(2, 3, 4, 64, 64), Bc_cache=torch.zeros(2, 3, 4, 64, 128),
                 n_cache=torch.zeros(2, dtype=torch.int32), gates_in=torch.zeros(2, 5, 3, 4))
    cache[missing] = None
    with pytest.raises(ValueError, match=missing):
        hla.gdn_tree_decode(q, **t, **cache)
