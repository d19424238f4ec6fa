"""The gradient of the decays (la_prefill_backward's dlog_decay) where a loss lies on one side of a row, where
values do not cancel, and where inputs are not finite.

Bounds.  dg_t is a sum over pairs of a token in front of t and one at or behind it, so its magnitudes are below
those of either side's tokens.  With b_j = k_j . dk_j and c_j = q_j . dq_j, the tokens up to the end of t's piece (64
tokens at most), or those from its start on, give it: b and c of every token at most once, the piece's own pairs once
more (their magnitudes are below b's and c's), and the product of the two states at the side's end.  A token's
sum is off by `steps` (see la_util) of its magnitudes and different tokens' roundings are independent: the value is
off by 2 steps of the root of the side's sum of squares, of the smaller side's since the call takes that one."""
import numpy as np
import pytest
import torch

from gated_deltanet_hybrid_amd import hla
from gpu_util import note
from la_util import Case, U, steps
from oracle import la as ola

pytestmark = pytest.mark.gpu


def side(x):
    """The root of the smaller side's sum of squares for every token of one head."""
    a = {n: None if x[n] is None else np.abs(x[n]) for n in ("q", "k", "v", "dO", "dS", "S0")}
    d = ola.la_backward(a["q"], a["k"], a["v"], x["g"], a["dO"], a["dS"], a["S0"])
    _, M = ola.la_recurrent(a["q"], a["k"], a["v"], x["g"], a["S0"])
    n = len(x["g"])
    own = (a["k"] * d["dk"]).sum(-1) ** 2 + (a["q"] * d["dq"]).sum(-1) ** 2
    front = np.cumsum(own) + (0.0 if a["S0"] is None else np.sum(d["dS0"] * a["S0"]) ** 2)
    behind = np.cumsum(own[::-1])[::-1] + (0.0 if a["dS"] is None else np.sum(a["dS"] * M[-1]) ** 2)
    start = np.arange(n) // 64 * 64
    return np.sqrt(np.minimum(front[np.minimum(start + 63, n - 1)], behind[start]))


def grads(c, rounding=None):
    """(dg [B, T, H], its bounds) in float64; rounding: of a token's sums, where steps is too much."""
    out = np.zeros((2, c.B, c.T, c.H))
    for b, h, n, x in c.rows():
        if n:
            out[0, b, :n, h] = ola.la_backward(x["q"], x["k"], x["v"], x["g"], x["dO"], x["dS"], x["S0"])["dg"]
            out[1, b, :n, h] = 2 * (rounding or steps(2 * c.T + 4 * c.dk)) * side(x) + 1e-37
    return out


def run(c, times=1, **kw):
    """The call on `times` copies of the batch (many rows stay whole, few are cut into segments); the first copy's gradients."""
    many = lambda t: None if t is None else t.repeat(times, *[1] * (t.dim() - 1)).contiguous()  # noqa: E731
    q, k, v, g = c.args()
    rest = {n: many(t) for n, t in c.kw().items()}
    d = hla.la_prefill_backward(many(q), many(k), many(v), g if g.dim() == 1 else many(g), many(c.device("dO")),
                                dS_final=many(c.device("dS")), **rest, **kw)
    torch.cuda.synchronize()
    return d


def spread(c, rate):
    """Decays of `rate` to 3 `rate` a token in place of the drawn ones."""
    r = np.random.default_rng(7)
    c.g_ = torch.from_numpy((-rate * (1.0 + 2.0 * r.random(tuple(c.g_.shape)))).astype(np.float32))


WHERE = {"first": lambda T: slice(0, 40), "last": lambda T: slice(T - 40, T), "all": lambda T: slice(0, T)}


def losses(c, where):
    """A loss on these tokens alone."""
    at, dO = WHERE[where](c.T), torch.zeros_like(c.dO_)
    dO[:, at] = c.dO_[:, at]
    c.dO_ = dO
    if where != "all":
        c.dS_ = None


# (B, T, H, Hk, dk, dv, dtype, start), copies of the batch
ROWS = [((2, 700, 1, 1, 64, 64, "f32", True), 270), ((1, 500, 1, 1, 64, 128, "f32", False), 540),
        ((2, 700, 2, 1, 128, 64, "bf16", True), 140), ((1, 900, 1, 1, 128, 128, "bf16", False), 540),
        ((1, 32 * 40 + 3, 1, 1, 64, 64, "f32", True), 1), ((1, 64 * 40 - 5, 1, 1, 64, 64, "bf16", False), 1)]


@pytest.mark.parametrize("rate", [0.02, 0.1, 0.5])
@pytest.mark.parametrize("where", list(WHERE))
@pytest.mark.parametrize("shape,times", ROWS, ids=str)
def test_a_loss_on_one_side(shape, times, where, rate):
    """Only some tokens have a loss: the others' gradients shrink with every token between, and so must their errors."""
    note(f"dlog_decay {shape} x {times} {where} {rate}")
    *a, start = shape
    c = Case(*a, start=start, seed=31)
    spread(c, rate)
    losses(c, where)
    ref, lim = grads(c)
    d = run(c, times)
    got = d["dlog_decay"]
    assert torch.equal(got, got[:c.B].repeat(times, 1, 1))
    err = np.abs(got[:c.B].double().cpu().numpy() - ref)
    worst = float(np.max(err / lim))
    note(f"  share of the bound {worst:.3f}")
    assert worst <= 1.0, (worst, np.argwhere(err > lim)[:4].tolist(), int((err > lim).sum()))
    if start:  # the same bits where the initial state's gradient is not asked for
        e = run(c, times, want_dS0=False)
        assert e["dS0"] is None and torch.equal(e["dlog_decay"], got)


@pytest.mark.parametrize("where", list(WHERE))
@pytest.mark.parametrize("shape,times", ROWS, ids=str)
def test_one_decay_a_head_of_values_that_do_not_cancel(shape, times, where):
    """Where no term is negative a sum is its magnitude, and the bounds on the tokens say something of their sum.  A
    float32 sum of n such terms has partial sums that grow to s: 6 standard deviations of their roundings are
    6 sqrt(n / 9) 2^-24 s, with n the state's width and height and the tokens that a decay of 0.05 leaves."""
    note(f"dlog_decay a head {shape} x {times} {where}")
    *a, start = shape
    c = Case(*a, per_head=True, start=start, seed=32)
    spread(c, 0.05)
    for n in ("q_", "k_", "v_", "dO_", "S0_", "dS_"):
        t = getattr(c, n)
        setattr(c, n, None if t is None else t.abs())
    losses(c, where)
    terms = c.dk + c.dv + 16 / 0.05
    ref, lim = (x.sum(1).sum(0) for x in grads(c, (6 * np.sqrt(terms / 9) + 24) * U))
    assert (lim < 1e-4 * ref).all()
    got = run(c, times)["dlog_decay"].double().cpu().numpy() / times
    note(f"  relative error {np.max(np.abs(got - ref) / ref):.2e}, share of the bound {np.max(np.abs(got - ref) / lim):.3f}")
    assert (np.abs(got - ref) <= lim).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("times", [1, 300])
@pytest.mark.parametrize("what", ["k", "v"])
def test_a_key_that_is_not_finite_leaves_earlier_tokens(dtype, times, what):
    """dg_t sums keys and values in front of t: one behind t's piece does not reach it."""
    note(f"dlog_decay not finite {dtype} {times} {what}")
    c = Case(2, 640, 1, 1, 64, 64, dtype, seed=33)
    spread(c, 0.02)
    ref, lim = grads(c)
    at, piece = 400, 64 if dtype == "bf16" else 32
    getattr(c, what + "_")[0, at, 0, 3] = float("nan")
    got = run(c, times)["dlog_decay"][:2].double().cpu().numpy()
    first = at // piece * piece
    assert (np.abs(got - ref)[0, :first] <= lim[0, :first]).all()
    assert (np.abs(got - ref)[1] <= lim[1]).all()
    assert np.isnan(got[0, at + 1:]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("times", [1, 300])
@pytest.mark.parametrize("what", ["q", "dO"])
def test_a_query_that_is_not_finite_leaves_later_tokens(dtype, times, what):
    note(f"dlog_decay not finite {dtype} {times} {what}")
    c = Case(2, 640, 1, 1, 64, 64, dtype, seed=34)
    spread(c, 0.02)
    ref, lim = grads(c)
    at, piece = 200, 64 if dtype == "bf16" else 32
    getattr(c, what + "_")[0, at, 0, 3] = float("nan")
    got = run(c, times)["dlog_decay"][:2].double().cpu().numpy()
    behind = (at // piece + 1) * piece
    assert (np.abs(got - ref)[0, behind:] <= lim[0, behind:]).all()
    assert (np.abs(got - ref)[1] <= lim[1]).all()
    assert np.isnan(got[0, 1:at + 1]).all()


def test_rows_of_the_most_segments():
    """A row whose segments number 128 of more than 64 pieces each, were they not cut further: windows of it against their
    own tokens (what is 2000 tokens away has decayed to nothing), and a key that is not finite behind them."""
    note("dlog_decay of a long row")
    T = 32 * 64 * 128 + 5000
    r = torch.Generator().manual_seed(9)
    q, k, v, dO = (torch.randn(1, T, 1, 64, generator=r) for _ in range(4))
    q, k = (torch.nn.functional.normalize(x, dim=-1) for x in (q, k))
    g = -0.05 - 0.1 * torch.rand(1, T, 1, generator=r)
    bad = 32 * 2000 + 1900
    windows = [0, 32 * 65 * 7 - 1000, bad // 32 * 32 - 2000, T - 2000]

    def check(got, lo):
        a, b = max(lo - 2000, 0), min(lo + 4000, T)
        x = dict(zip(("q", "k", "v", "dO"), (y[0, a:b, 0].double().numpy() for y in (q, k, v, dO))))
        x.update(g=g[0, a:b, 0].double().numpy(), dS=None, S0=None)
        ref = ola.la_backward(x["q"], x["k"], x["v"], x["g"], x["dO"])["dg"]
        lim = 2 * steps(2 * 2000 + 4 * 64) * side(x) + 1e-37
        at = slice(lo - a, lo - a + 2000)
        assert (np.abs(got[lo:lo + 2000] - ref[at]) <= lim[at]).all(), lo

    call = lambda: hla.la_prefill_backward(*(x.cuda() for x in (q, k, v, g, dO)))["dlog_decay"][0, :, 0].double().cpu().numpy()  # noqa: E731
    got = call()
    for lo in windows:
        check(got, lo)
    k[0, bad, 0, 3] = float("nan")
    got = call()
    assert np.isfinite(got[:bad // 32 * 32]).all() and np.isnan(got[bad + 1:]).all()
