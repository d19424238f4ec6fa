"""Decays that clear the state of linear attention: below float32's smallest normal number, -inf included."""
import pytest
import torch

from gated_deltanet_hybrid_amd import hla
from gpu_util import note
from la_util import Case

pytestmark = pytest.mark.gpu

CLEARS = [-87.5, -95.0, -103.0, -104.5, -9999.0, -1e5, -float("inf")]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("T", [1, 40, 700])
def test_a_cleared_state_is_forgotten(dtype, per_head, T):
    """Whatever stood in the state has no effect behind such a decay, and no gradient passes it."""
    note(f"la clears {dtype} {per_head} {T}")
    for g in CLEARS:
        c = Case(2, T, 2, 1, 64, 64, dtype, per_head=per_head, seed=51)
        q, k, v, _ = c.args()
        gg = torch.full((2,), g, device="cuda") if per_head else torch.full((2, T, 2), -0.1, device="cuda")
        at = [0] if per_head else sorted({0, T // 2, T - 1})
        if not per_head:
            gg[:, at] = g
        S0 = 1e20 * c.device("S0")
        o, S = hla.la_prefill(q, k, v, gg, S0=S0)
        o2, S2 = hla.la_prefill(q, k, v, gg)
        assert torch.equal(o, o2) and torch.equal(S, S2), g
        d = hla.la_prefill_backward(q, k, v, gg, c.device("dO"), dS_final=1e20 * c.device("dS"), S0=S0)
        assert (d["dS0"] == 0).all(), g
        cleared = d["dlog_decay"] if per_head else d["dlog_decay"][:, at]
        assert (cleared == 0).all(), (g, cleared)
        one = [x[:, 0].contiguous() for x in (q, k, v)] + [gg if per_head else gg[:, 0].contiguous()]
        A, B = S0.clone(), torch.zeros_like(S0)
        assert torch.equal(hla.la_decode(*one, A), hla.la_decode(*one, B)) and torch.equal(A, B), g


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_smallest_decay_that_does_not(dtype):
    """exp(-87) is a normal number: a state of 2^100 shows behind it."""
    note(f"la keeps {dtype}")
    c = Case(1, 1, 1, 1, 64, 64, dtype, seed=52)
    q, k, v, _ = c.args()
    g, S0 = torch.full((1, 1, 1), -87.0, device="cuda"), 2.0 ** 100 * c.device("S0")
    _, S = hla.la_prefill(q, 0 * k, v, g, S0=S0)
    want = S0.double() * torch.exp(torch.tensor(-87.0, dtype=torch.float64, device="cuda"))
    # exp: its argument in base 2 is rounded to float32 (126 half steps of 2^-24 ln 2 a unit), and the result once more
    assert ((S.double() - want).abs() <= (126 + 4) * 2.0 ** -24 * want.abs()).all()
