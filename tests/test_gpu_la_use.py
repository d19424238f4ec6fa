"""Linear attention and trees of drafted tokens as programs use them: in captured graphs, on other streams,
in place, in windows of longer buffers, in pieces, with guard bands, with numbers that are not finite."""
import numpy as np
import pytest
import torch

from gated_deltanet_hybrid_amd import hla
from gpu_util import note
from la_util import Case, bound, check, steps
from test_gpu_tree import call, make, num, reference
from test_gpu_tree import check as check_tree

pytestmark = pytest.mark.gpu


def bits(x):
    return x.view(torch.int16 if x.dtype == torch.bfloat16 else torch.int32)


def same(a, b):
    return torch.equal(bits(a), bits(b))


# one segment, and several (two rows of 40 pieces)
SHAPES = [(3, 90, 4, 2, 64, 128, "bf16"), (1, 64 * 40 - 9, 2, 1, 128, 64, "bf16"), (1, 32 * 40 - 9, 2, 2, 64, 64, "f32")]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_calls_repeat_their_bits(shape):
    note(f"la determinism {shape}")
    c = Case(*shape, per_head=True)
    runs = []
    for _ in range(3):
        o, S = hla.la_prefill(*c.args(), **c.kw())
        d = hla.la_prefill_backward(*c.args(), c.device("dO"), dS_final=c.device("dS"), **c.kw())
        runs.append([o, S] + [d[k] for k in sorted(d)])
    for r in runs[1:]:
        assert all(same(a, b) for a, b in zip(runs[0], r))


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_final_state_in_place_of_the_initial_one(shape):
    note(f"la in place {shape}")
    c = Case(*shape)
    o, S = hla.la_prefill(*c.args(), **c.kw())
    S0 = c.device("S0").clone()
    o2, S2 = hla.la_prefill(*c.args(), S0=S0, S_final=S0)
    assert S2.data_ptr() == S0.data_ptr() and same(S, S2) and same(o, o2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("per_head", [False, True])
def test_a_prompt_in_parts_then_tokens(dtype, per_head):
    """A prompt in two calls and its last tokens one by one, against the whole in float64."""
    note(f"la serving run {dtype} {per_head}")
    B, T, H, Hk, dk, dv = 2, 180, 4, 2, 128, 64
    c = Case(B, T, H, Hk, dk, dv, dtype, per_head=per_head)
    q, k, v, g = c.args()
    gg = lambda s: g if per_head else g[:, s]  # noqa: E731
    o1, S = hla.la_prefill(q[:, :70], k[:, :70], v[:, :70], gg(slice(0, 70)), S0=c.device("S0"))
    o2, S = hla.la_prefill(q[:, 70:172], k[:, 70:172], v[:, 70:172], gg(slice(70, 172)), S0=S)
    outs = [o1, o2]
    for t in range(172, T):
        one = hla.la_decode(*(x[:, t].contiguous() for x in (q, k, v)), g if per_head else g[:, t].contiguous(), S)
        outs.append(one[:, None])
    ro, rS = c.forward()
    check(torch.cat(outs, 1), ro[0], ro[1], dtype, T + 2 * dk, "o")
    check(S, rS[0], rS[1], "f32", T + 2 * dk, "S")


def test_windows_of_longer_buffers():
    note("la windows")
    c = Case(2, 100, 4, 2, 128, 128, "bf16", ld_T=300)
    full = [getattr(c, n + "_").cuda() for n in ("q", "k", "v", "g")]
    for lo in (0, 1, 130, 200):
        part = [x[:, lo:lo + 100] for x in full]
        o, S = hla.la_prefill(*part, S0=c.device("S0"))
        o2, S2 = hla.la_prefill(*(x.contiguous() for x in part), S0=c.device("S0"))
        assert same(o, o2) and same(S, S2)
        a = hla.la_prefill_backward(*part, c.device("dO"), S0=c.device("S0"))
        b = hla.la_prefill_backward(*(x.contiguous() for x in part), c.device("dO"), S0=c.device("S0"))
        assert all(same(a[k], b[k]) for k in a)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_graph_replays(shape):
    """Captured with static inputs and replayed on new ones, eager work in between; every replay has the
    eager call's bits."""
    note(f"la graph {shape}")
    c = Case(*shape)
    q, k, v, g = c.args()
    S0, dO, dS = c.device("S0"), c.device("dO"), c.device("dS")
    B, T, H = v.shape[:3]
    lens = torch.full((B,), T, dtype=torch.int32, device="cuda")
    St = S0.clone()
    step = [x[:, 0].contiguous() for x in (q, k, v, g)]

    def work():
        o, S = hla.la_prefill(q, k, v, g, S0=S0, lens=lens)
        d = hla.la_prefill_backward(q, k, v, g, dO, dS_final=dS, S0=S0, lens=lens)
        return [o, S, hla.la_decode(*step, St)] + [d[n] for n in sorted(d)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = work()
    for i in range(4):
        other = Case(*shape, seed=10 + i)
        for name, to in (("q", q), ("k", k), ("v", v), ("g", g), ("S0", S0), ("dO", dO), ("dS", dS)):
            to.copy_(other.device(name))
        for a, b in zip(step, (q, k, v, g)):
            a.copy_(b[:, 0])
        lens.fill_(max(T - 7 * i, 0))
        St.copy_(S0)
        want = [x.clone() for x in work()]
        St.copy_(S0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(outs, want)), i


def test_two_streams_at_once():
    note("la two streams")
    cases = [Case(1, 64 * 30, 2, 2, 128, 128, "bf16", seed=s) for s in (1, 2)]
    want = [hla.la_prefill(*c.args(), **c.kw()) for c in cases]
    ins = [(c.args(), c.kw()) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(hla.la_prefill(*ins[i][0], **ins[i][1]))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(same(w[0], o) and same(w[1], S) for o, S in g)


@pytest.mark.parametrize("shape", SHAPES + [(2, 33, 3, 1, 64, 128, "f32"), (2, 65, 6, 2, 128, 64, "bf16")], ids=str)
def test_guard_bands(shape):
    """Outputs and a workspace of the asked size between bands that stay as they were."""
    note(f"la guards {shape}")
    c = Case(*shape, lens=[shape[1] - 3] + [shape[1]] * (shape[0] - 1))
    q, k, v, g = c.args()
    B, T, H, Hk, dk, dv = shape[:6]
    band = 4096

    def guarded(n, dtype):
        size = n * torch.tensor([], dtype=dtype).element_size()
        raw = torch.full((size + 2 * band,), 0xA5, dtype=torch.uint8, device="cuda")
        return raw, raw[band:band + size].view(dtype)

    raws = []

    def take(shape_, dtype):
        raw, x = guarded(int(np.prod(shape_)), dtype)
        raws.append(raw)
        return x.view(*shape_)

    n = hla.la_workspace_bytes(hla.LA_PREFILL, q, k, v, g)
    ws = take((max(n, 16),), torch.uint8)
    o, S = take((B, T, H, dv), v.dtype), take((B, H, dk, dv), torch.float32)
    hla.la_prefill(q, k, v, g, o=o, S_final=S, ws=ws if n else None, **c.kw())
    import ctypes
    n = hla.la_workspace_bytes(hla.LA_PREFILL_BACKWARD, q, k, v, g)
    ws2 = take((n,), torch.uint8)
    d = dict(dq=take((B, T, Hk, dk), v.dtype), dk=take((B, T, Hk, dk), v.dtype), dv=take((B, T, H, dv), v.dtype),
             dg=take((B, T, H), torch.float32), dS0=take((B, H, dk, dv), torch.float32))
    dims, dev = hla._la_inputs(q, k, v, g, c.kw()["lens"])
    lens, dO, dS, S0 = c.kw()["lens"], c.device("dO"), c.device("dS"), c.device("S0")
    p = lambda t: t.data_ptr()  # noqa: E731
    hla._call("hla_la_prefill_backward", dev, ctypes.byref(dims), p(q), p(k), p(v), p(g), p(lens), p(S0), p(dO), p(dS),
              p(d["dq"]), p(d["dk"]), p(d["dv"]), p(d["dg"]), p(d["dS0"]), p(ws2), n)
    torch.cuda.synchronize()
    for raw in raws:
        assert (raw[:band] == 0xA5).all() and (raw[-band:] == 0xA5).all()
    e = hla.la_prefill_backward(q, k, v, g, dO, dS_final=dS, **c.kw())
    assert same(d["dq"], e["dq"]) and same(d["dk"], e["dk"]) and same(d["dv"], e["dv"]) and same(d["dS0"], e["dS0"])
    assert same(d["dg"], e["dlog_decay"])


def test_offsets_past_32_bits():
    """A batch whose tensors pass 2^31 elements: its last row alone gives the same bits."""
    note("la large offsets")
    B, T, H, d = 9, 125000, 16, 128  # 2.3e9 elements a tensor
    k = torch.empty(B, T, H, d, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    gen = torch.Generator(device="cuda").manual_seed(3)
    for x in (k, v):
        x.zero_()
        x[-1].normal_(generator=gen)
    g = torch.full((B, T, H), -0.05, device="cuda")
    lens = torch.tensor([0] * (B - 1) + [T], dtype=torch.int32, device="cuda")
    o, S = hla.la_prefill(k, k, v, g, lens=lens)
    tail = slice(T - 6400, T)  # exp(-0.05 * 6400) is nothing: the last tokens do not know the first
    o1, S1 = hla.la_prefill(k[-1:, tail].contiguous(), k[-1:, tail].contiguous(), v[-1:, tail].contiguous(),
                            g[-1:, tail].contiguous())
    a, b = o[-1, -640:].float(), o1[0, -640:].float()
    assert (a - b).abs().max() <= 2.0 ** -7 * b.abs().max()
    assert (S[-1] - S1[0]).abs().max() <= 64 * steps(2 * 6400) * S1.abs().max()
    assert (o[:-1].view(torch.int16).amax() == 0) and (S[:-1] == 0).all()


def test_tokens_behind_a_row_are_not_read():
    note("la behind the row")
    for dtype in ("bf16", "f32"):
        c = Case(3, 100, 2, 2, 64, 64, dtype, lens=[63, 0, 65])
        o, S = hla.la_prefill(*c.args(), **c.kw())
        d = hla.la_prefill_backward(*c.args(), c.device("dO"), dS_final=c.device("dS"), **c.kw())
        for b, n in enumerate(c.lens):
            for name in ("q_", "k_", "v_", "g_", "dO_"):
                getattr(c, name)[b, n:] = float("nan") if b else float("inf")
        o2, S2 = hla.la_prefill(*c.args(), **c.kw())
        e = hla.la_prefill_backward(*c.args(), c.device("dO"), dS_final=c.device("dS"), **c.kw())
        assert same(o, o2) and same(S, S2) and all(same(d[k], e[k]) for k in d)
        for b, n in enumerate(c.lens):
            assert (o2[b, n:] == 0).all() and (e["dq"][b, n:] == 0).all() and (e["dlog_decay"][b, n:] == 0).all()


def test_a_nan_stays_behind_its_piece():
    note("la nan")
    c = Case(1, 200, 2, 2, 64, 64, "bf16")
    q, k, v, g = c.args()
    g = torch.full_like(g, -0.1)
    o, _ = hla.la_prefill(q, k, v, g)
    v[0, 100, 0, 5] = float("nan")
    o2, S2 = hla.la_prefill(q, k, v, g)
    assert same(o[:, :64], o2[:, :64]) and same(o[:, :, 1], o2[:, :, 1])
    assert torch.isnan(o2[0, 100:, 0, 5]).all() and torch.isnan(S2[0, 0, :, 5]).all()


@pytest.mark.parametrize("per_head", [False, True])
def test_gradients_against_differences(per_head):
    """The change of L = sum(o dO) + sum(S dS) along a direction against the gradient's, float32.  The
    difference is off by the rounding of both values of L (their bound over the step) and by the step's
    third-order term, which the float64 recurrence's own difference shows."""
    note(f"la differences {per_head}")
    B, T, H, Hk, dk, dv = 1, 70, 2, 1, 64, 64
    c = Case(B, T, H, Hk, dk, dv, "f32", per_head=per_head)
    if not per_head:
        c.g_ = c.g_.clamp(min=-3.0)  # finite logarithms: a step away from -inf is none
    r = np.random.default_rng(5)
    d = hla.la_prefill_backward(*c.args(), c.device("dO"), dS_final=c.device("dS"), **c.kw())
    eps = 2.0 ** -6

    def gpu_loss():
        o, S = hla.la_prefill(*c.args(), **c.kw())
        return float((o.double() * c.device("dO").double()).sum() + (S.double() * c.device("dS").double()).sum())

    def ref_loss():
        (o, om), (S, Sm) = c.forward()
        dO, dS = c.dO_.double().numpy(), c.dS_.double().numpy()
        return np.sum(o * dO) + np.sum(S * dS), np.sum(om * np.abs(dO)) + np.sum(Sm * np.abs(dS))

    ref = c.backward()
    for name, key in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dlog_decay"), ("S0", "dS0")):
        t = getattr(c, name + "_")
        keep = t.clone()
        delta = torch.from_numpy(r.choice([-1.0, 1.0], size=tuple(t.shape)).astype(np.float32))
        if name == "g":
            delta *= 0.25
        sides = []
        for s in (eps, -eps):
            setattr(c, name + "_", keep + s * delta)
            sides.append((gpu_loss(), *ref_loss()))
        setattr(c, name + "_", keep)
        diff, exact = ((sides[0][i] - sides[1][i]) / (2 * eps) for i in (0, 1))
        along = float((d[key].double().cpu() * delta.double()).sum())
        want = float(np.sum(ref[key][0] * delta.double().numpy()))
        mag = max(s[2] for s in sides)
        # a float32 step: keep + eps delta is itself rounded to half a step of the value
        lim = steps(T + 2 * dk) * mag / eps + abs(exact - want) + 2.0 ** -24 * mag / eps
        lim += steps(2 * T + 4 * dk) * float(np.sum(ref[key][1]))
        assert abs(diff - along) <= lim, (name, diff, along, lim)
        if not (name == "g" and per_head):  # the bound says something (of a sum over a row's tokens it says less)
            assert lim < 0.2 * abs(along) + 0.05 * float(np.sqrt(np.sum(ref[key][0] ** 2))) * np.sqrt(delta.numel()), name


# ------------------------------------------------------------------------------- trees
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tree_decode_changes_nothing_and_repeats(dtype):
    note(f"tree inputs stay {dtype}")
    x = make(2, 20, 2, 128, 64, dtype, 4, 3, seed=11)
    d = {n: t.cuda() for n, t in x.items()}
    before = {n: t.clone() for n, t in d.items()}
    rest = {m: d[m] for m in ("At_cur", "At_cache", "Bc_cache", "reps_cache", "n_cache")}
    outs = [hla.gdn_tree_decode(d["q"], d["k"], d["v"], d["beta"], d["alpha"], d["parent"], d["S_cur"], tau=0.3, **rest)
            for _ in range(3)]
    assert all(torch.equal(d[n], before[n]) for n in d)
    assert all(same(outs[0], o) for o in outs[1:])


@pytest.mark.parametrize("n", [7, 40])
def test_tree_graph_replays(n):
    note(f"tree graph n={n}")
    x = make(2, n, 2, 64, 128, "bf16", 5, 2, seed=12)
    d = {m: t.cuda() for m, t in x.items()}
    node = torch.tensor([n - 1, 0], dtype=torch.int32, device="cuda")
    commit = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    live = ("S_cur", "At_cur", "At_cache", "Bc_cache", "n_cache")
    start = {m: d[m].clone() for m in live}

    def work():
        o = hla.gdn_tree_decode(d["q"], d["k"], d["v"], d["beta"], d["alpha"], d["parent"], tau=0.3,
                                reps_cache=d["reps_cache"], **{m: d[m] for m in live})
        hla.gdn_tree_accept(d["k"], d["v"], d["beta"], d["alpha"], d["parent"], node, commit=commit, **{m: d[m] for m in live})
        return o

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = work()
    for i in range(4):
        fresh = make(2, n, 2, 64, 128, "bf16", 5, 2, seed=30 + i)
        for m in ("q", "k", "v", "beta", "alpha", "parent"):
            d[m].copy_(fresh[m])
        start["n_cache"].fill_(i)
        for m in live:
            d[m].copy_(start[m])
        want = work().clone()
        after = {m: d[m].clone() for m in live}
        for m in live:
            d[m].copy_(start[m])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert same(o, want) and all(torch.equal(d[m], after[m]) for m in live), i


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("what,value", [("k", float("nan")), ("v", float("inf")), ("q", float("nan")), ("alpha", float("nan")),
                                        ("beta", float("inf"))])
def test_what_is_not_finite_stays_in_its_branch(dtype, what, value):
    note(f"tree not finite {dtype} {what}")
    x = make(1, 12, 1, 64, 64, dtype, 3, 2, seed=13)
    x["parent"][0] = torch.tensor([-1, 0, 0, 1, 2, 3, 4, -1, 7, 8, 2, 5], dtype=torch.int32)
    bad, below = 2, {2, 4, 6, 10}
    clean = reference(x, 0.3)[0]
    x[what][0, bad] = value
    o = call(x, tau=0.3).cpu()
    fine = [i for i in range(12) if i not in (below if what != "q" else {2})]
    ref = clean[:, :, fine]
    check_tree(o[:, fine], ref, 12 + 64 + 3 * 64, "nodes outside the branch")
    for i in (below if what != "q" else {2}):
        assert not torch.isfinite(o[0, i]).all(), i


@pytest.mark.parametrize("Bs,H,n,n_cap", [(1, 3, 9, 1024), (40, 16, 33, 2), (300, 2, 17, 3), (60, 2, 40, 3)])
def test_tree_few_and_many_rows(Bs, H, n, n_cap):
    """The forms that the sizes choose: one launch or two in front, one or two chunks ahead, one to four
    tiles of nodes a workgroup.  Rows drawn from a few, so that the reference is quick."""
    note(f"tree forms {Bs} {H} {n} {n_cap}")
    x = make(1, n, 1, 64, 64, "bf16", n_cap, 2, seed=14)
    big = {}
    for m, t in x.items():
        reps = [1] * t.dim()
        reps[0] = Bs
        if m not in ("parent", "n_cache"):
            reps[2 if m in ("q", "k", "v", "beta", "alpha") else 1] = H
        big[m] = t.repeat(*reps)
    gates = torch.empty(Bs, n, H, n_cap, device="cuda")
    o = call(big, tau=0.3, gates_out=gates)
    assert all(same(o[b, :, h], o[0, :, 0]) for b, h in ((0, 0), (Bs - 1, H - 1), (Bs // 2, 0)))
    ref, rg = reference(x, 0.3)
    assert not (np.abs(rg - 0.3) < 1e-5).any()
    # over a thousand chunks the magnitudes overflow and bound nothing: the maps here keep z's length, so a
    # chunk's roundings stay relative to the result, and as many of them add up as there are terms
    terms = n + 64 + n_cap * 64
    err = num(o[:1, :, :1].cpu()) - ref[0]
    assert np.linalg.norm(err) <= steps(terms) * np.linalg.norm(ref[0])
    if n_cap < 100:
        check_tree(o[:1, :, :1], ref, terms, "o")
    assert np.abs(num(gates[:1, :, :1].cpu()) - rg).max() < 1e-4


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_absent_nodes_are_zero_over_any_live_state(dtype):
    note(f"tree absent {dtype}")
    x = make(1, 20, 2, 64, 128, dtype, 2, 2, seed=15)
    x["parent"][0, 17:] = -2
    x["parent"][0, 4] = 4
    x["S_cur"][0, :, 3, 5] = float("inf")
    x["At_cur"][0, :, 7, 9] = float("nan")
    o = call(x, tau=0.3)
    assert (o[0, 17:] == 0).all() and (o[0, 4] == 0).all()
    assert not torch.isfinite(o[0, 0]).all()


# few distinct rows, repeated: (rows, T, repeated) so that rows stay whole, are cut into segments of several
# pieces, and into as many segments as there are
@pytest.mark.parametrize("B,T,times,dk,dv,dtype,lens", [
    (3, 200, 180, 64, 128, "f32", None), (3, 330, 180, 128, 64, "bf16", [330, 0, 100]), (2, 650, 24, 128, 128, "bf16", None),
    (2, 400, 40, 64, 64, "f32", [400, 37]), (1, 32 * 260 + 3, 1, 64, 64, "f32", None), (1, 64 * 150, 1, 64, 64, "bf16", None)])
def test_rows_whole_and_cut(B, T, times, dk, dv, dtype, lens):
    note(f"la rows {B} {T} {times} {dk} {dv} {dtype}")
    c = Case(B, T, 1, 1, dk, dv, dtype, lens=lens, seed=21)
    many = lambda t: None if t is None else t.repeat(times, *[1] * (t.dim() - 1)).contiguous()  # noqa: E731
    q, k, v, g = map(many, c.args())
    kw = {n: many(t) for n, t in c.kw().items()}
    dO, dS = many(c.device("dO")), many(c.device("dS"))
    o, S = hla.la_prefill(q, k, v, g, **kw)
    d = hla.la_prefill_backward(q, k, v, g, dO, dS_final=dS, **kw)
    for t in (o, S, *d.values()):
        assert torch.equal(t, many(t[:B]))
    (ro, rS), rd, n = c.forward(), c.backward(), T + 2 * dk
    check(o[:B], ro[0], ro[1], dtype, n, "o")
    check(S[:B], rS[0], rS[1], "f32", n, "S_final")
    for m, ref in rd.items():
        check(d[m][:B], ref[0], ref[1], dtype if m in ("dq", "dk", "dv") else "f32", 2 * T + 4 * dk, m)
