"""hla_timing_enable sees linear attention and trees of drafted tokens, and changes none of their results."""
import pytest
import torch

from gated_deltanet_hybrid_amd import hla
from gpu_util import note
from la_util import Case
from test_gpu_tree import make

pytestmark = pytest.mark.gpu


def test_calls_are_timed():
    note("timing of linear attention and trees")
    c = Case(1, 900, 2, 1, 64, 64, "bf16")
    q, k, v, g = c.args()
    one = [x[:, 0].contiguous() for x in (q, k, v, g)]
    d = {n: t.cuda() for n, t in make(2, 9, 2, 64, 64, "bf16", 3, 2).items()}
    tree = [d[n] for n in ("k", "v", "beta", "alpha", "parent")]
    cache = {n: d[n] for n in ("At_cur", "At_cache", "Bc_cache", "n_cache")}
    node = torch.full((2,), -1, dtype=torch.int32, device="cuda")

    def work():
        S = c.device("S0").clone()
        out = [*hla.la_prefill(q, k, v, g, S0=c.device("S0")), hla.la_decode(*one, S), S]
        out += hla.la_prefill_backward(q, k, v, g, c.device("dO"), S0=c.device("S0")).values()
        out.append(hla.gdn_tree_decode(d["q"], *tree, d["S_cur"], reps_cache=d["reps_cache"], **cache))
        hla.gdn_tree_accept(*tree, node, d["S_cur"], **cache)
        return out

    want = work()
    hla.timing_enable(True)
    try:
        got = work()
        for kind, calls in ((hla.KERNEL_LA, 2), (hla.KERNEL_BWD_LA, 1), (hla.KERNEL_TREE, 2)):
            ms, n = hla.timing_read(kind)
            assert n == calls and 0.0 < ms < 1e3, kind
        for kind in range(hla.KERNEL_LA):
            assert hla.timing_read(kind)[1] == 0
    finally:
        hla.timing_enable(False)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
