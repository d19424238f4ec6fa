"""Linear attention with a decay for each head (la_prefill, la_prefill_backward, la_decode) against
the float64 recurrence."""
import numpy as np
import pytest
import torch

from gated_deltanet_hybrid_amd import hla
from gpu_util import note
from la_util import Case, bound, check

pytestmark = pytest.mark.gpu

# (B, T, H, Hk, dk, dv, dtype, options)
PREFILL = [
    (1, 1, 1, 1, 64, 64, "bf16", {}),
    (1, 1, 2, 2, 128, 128, "f32", dict(start=False)),
    (2, 31, 2, 1, 64, 128, "f32", {}),
    (1, 32, 2, 2, 128, 64, "f32", dict(per_head=True)),
    (1, 33, 3, 3, 128, 128, "f32", {}),
    (2, 63, 2, 2, 128, 128, "bf16", dict(start=False)),
    (1, 64, 2, 2, 64, 128, "bf16", dict(per_head=True)),
    (1, 65, 4, 2, 128, 64, "bf16", {}),
    (3, 150, 4, 1, 64, 64, "bf16", dict(lens=[150, 0, 1])),
    (4, 150, 2, 2, 128, 128, "f32", dict(lens=[64, 65, -3, 1000])),
    (2, 200, 2, 2, 128, 128, "bf16", dict(ld_T=333, lens=[200, 64])),
    (2, 130, 2, 1, 64, 64, "f32", dict(ld_T=131)),
    (1, 256, 2, 2, 128, 128, "bf16", dict(decay="fast")),
    (1, 256, 2, 2, 128, 128, "f32", dict(decay="fast")),
    (1, 300, 2, 2, 64, 64, "bf16", dict(decay="none", start=False)),
    # few rows, long: segments (bf16 pieces of 64 tokens, 8 and more to a segment; float32 32)
    (1, 64 * 33 + 7, 2, 1, 64, 64, "bf16", {}),
    (2, 64 * 17, 1, 1, 128, 128, "bf16", dict(lens=[700, 64 * 17], per_head=True)),
    (1, 32 * 35 + 1, 1, 1, 64, 128, "f32", dict(lens=[900])),
    (1, 32 * 16, 1, 1, 128, 64, "f32", dict(decay="none")),
]


@pytest.mark.parametrize("case", PREFILL, ids=lambda c: "-".join(map(str, c)))
def test_prefill(case):
    *a, kw = case
    note(f"la_prefill {case}")
    c = Case(*a, **kw)
    o, S = hla.la_prefill(*c.args(), **c.kw())
    torch.cuda.synchronize()
    ro, rS = c.forward()
    n = c.T + 2 * c.dk
    w = [check(o, ro[0], ro[1], c.dtype, n, "o"), check(S, rS[0], rS[1], "f32", n, "S_final")]
    assert o.dtype == c.args()[2].dtype
    # the state alone: the same numbers, and without q
    _, S1 = hla.la_prefill(None, *c.args()[1:], want_o=False, **c.kw())
    check(S1, rS[0], rS[1], "f32", n, "S_final alone")
    o1, none = hla.la_prefill(*c.args(), want_state=False, **c.kw())
    assert none is None and torch.equal(o, o1)
    note(f"  share of the bounds: o {w[0]:.3f} S {w[1]:.3f}")


@pytest.mark.parametrize("case", PREFILL, ids=lambda c: "-".join(map(str, c)))
def test_backward(case):
    *a, kw = case
    note(f"la_prefill_backward {case}")
    c = Case(*a, **kw)
    d = hla.la_prefill_backward(*c.args(), c.device("dO"), dS_final=c.device("dS"), **c.kw())
    torch.cuda.synchronize()
    ref = c.backward()
    n = 2 * c.T + 4 * c.dk
    w = {}
    for name, (r, mag) in ref.items():
        w[name] = check(d[name], r, mag, c.dtype if name in ("dq", "dk", "dv") else "f32", n, name)
    note("  share of the bounds: " + " ".join(f"{k} {v:.3f}" for k, v in w.items()))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Bs,H,Hk,dk,dv,per_head", [(1, 1, 1, 64, 64, False), (3, 4, 2, 128, 64, True),
                                                    (2, 6, 1, 64, 128, False), (5, 2, 2, 128, 128, True)])
def test_decode_is_the_recurrence(dtype, Bs, H, Hk, dk, dv, per_head):
    note(f"la_decode {dtype} {Bs} {H} {Hk} {dk} {dv} {per_head}")
    T = 5
    c = Case(Bs, T, H, Hk, dk, dv, dtype, per_head=per_head)
    q, k, v, g = c.args()
    S = c.device("S0").clone()
    outs = []
    for t in range(T):
        outs.append(hla.la_decode(q[:, t].contiguous(), k[:, t].contiguous(), v[:, t].contiguous(),
                                  g if per_head else g[:, t].contiguous(), S))
    torch.cuda.synchronize()
    ro, rS = c.forward()
    check(S, rS[0], rS[1], "f32", T + 2, "S")
    got = torch.stack(outs, 1).float().cpu().numpy().astype(np.float64)
    lim = bound("f32", ro[0], ro[1], T + dk) + (2.0 ** -8 * np.abs(ro[0]) if dtype == "bf16" else 0.0)
    assert (np.abs(got - ro[0]) <= lim).all()


@pytest.mark.parametrize("dtype,T", [("bf16", 1), ("f32", 1), ("bf16", 200), ("f32", 200)])
def test_nothing_decays_in_front_of_a_zero_state(dtype, T):
    """The first token of a row meets a zero state: its decay has no effect, and its gradient is 0 and no
    rounding of something else."""
    note(f"la_prefill_backward from zero {dtype} {T}")
    c = Case(3, T, 2, 2, 64, 128, dtype, start=False, lens=[T, 1, 0])
    d = hla.la_prefill_backward(*c.args(), c.device("dO"), dS_final=torch.ones(3, 2, 64, 128, device="cuda"), **c.kw())
    assert (d["dlog_decay"][:, 0] == 0).all()
    assert (d["dlog_decay"][1:] == 0).all()
