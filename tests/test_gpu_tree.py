"""Trees of drafted tokens (gdn_tree_decode, gdn_tree_accept) against the float64 recurrence, node by
node: a node's answer is the decode step's after its own ancestors.

Bounds.  o is a sum of products; A, the same expressions over magnitudes (with + for every -), bounds its
terms.  The closed form takes the node's n - 1 ancestors, sums over dk and per chunk the map's dk: a
float32 sum of m terms is off by at most 6 sqrt(m / 3) 2^-24 A (six standard deviations of roundings of
half a step), decays and gates by 24 steps more.  z carries 24 bits through every chunk."""
import numpy as np
import pytest
import torch

from gated_deltanet_hybrid_amd import hla
from gpu_util import note

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def make(Bs, n, H, dk, dv, dtype, n_cap, n_rep, seed=0, shape="tree"):
    r = np.random.default_rng([seed, Bs, n, H, dk, dv])
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    f = lambda *s: torch.from_numpy(r.standard_normal(s).astype(np.float32))  # noqa: E731
    u = lambda *s: torch.from_numpy(r.random(s).astype(np.float32))  # noqa: E731
    x = dict(q=f(Bs, n, H, dk).to(td), k=torch.nn.functional.normalize(f(Bs, n, H, dk), dim=-1).to(td),
             v=f(Bs, n, H, dv).to(td), beta=u(Bs, n, H), alpha=0.7 + 0.3 * u(Bs, n, H))
    parent = np.full((Bs, n), -2, np.int32)
    for b in range(Bs):
        size = n if b == 0 else r.integers(0, n + 1)
        for i in range(size):
            parent[b, i] = i - 1 if shape == "chain" else -1 if shape == "star" else r.integers(max(-1, i - 5), i)
    x["parent"] = torch.from_numpy(parent)
    x["S_cur"], x["At_cur"] = 0.3 * f(Bs, H, dk, dv), torch.eye(dk) - 0.02 * u(Bs, H, dk, dk)
    if n_cap:
        x["At_cache"] = (torch.eye(dk) + 0.05 * f(Bs, H, n_cap, dk, dk) / dk ** 0.5).to(td)
        x["Bc_cache"] = (0.3 * f(Bs, H, n_cap, dk, dv)).to(td)
        x["reps_cache"] = (0.5 * f(Bs, H, n_cap, n_rep, dk)).to(td)
        count = r.integers(0, n_cap + 1, Bs)
        count[0] = n_cap
        x["n_cache"] = torch.from_numpy(count.astype(np.int32))
    return x


def num(t):
    return t.double().numpy()


def path_states(x, b, h):
    """Every present node's (M, At) in float64, -1 the live ones, with their bounds of magnitude."""
    k, v, beta, alpha = (num(x[n])[b, :, h] for n in ("k", "v", "beta", "alpha"))
    at = {-1: tuple(num(x[m])[b, h] for m in ("S_cur", "At_cur")) + tuple(np.abs(num(x[m])[b, h]) for m in ("S_cur", "At_cur"))}
    for i, p in enumerate(x["parent"][b].tolist()):
        if not (-1 <= p < i) or p not in at:
            continue
        M, A, Mm, Am = at[p]
        kk, km = k[i][:, None], np.abs(k[i])[:, None]
        M, A, Mm, Am = (alpha[i] * y for y in (M, A, Mm, Am))
        at[i] = (M - beta[i] * kk * (kk.T @ M) + beta[i] * kk * v[i][None], A - beta[i] * kk * (kk.T @ A),
                 Mm + beta[i] * km * (km.T @ Mm) + beta[i] * km * np.abs(v[i])[None], Am + beta[i] * km * (km.T @ Am))
    return at


def gates_of(x, b, h, i):
    q = num(x["q"])[b, i, h]
    s = num(x["reps_cache"])[b, h] @ q / np.sqrt(len(q))
    e = np.exp(s).mean(-1)
    return e / (1 + e)


def reference(x, tau, gates_in=None):
    """(o, magnitudes, gates) per node."""
    Bs, n, H, dk = x["q"].shape
    dv = x["v"].shape[-1]
    cached = "At_cache" in x
    o = np.zeros((2, Bs, n, H, dv))
    gates = np.zeros((Bs, n, H, x["At_cache"].shape[2] if cached else 0))
    for b in range(Bs):
        for h in range(H):
            for i, (M, A, Mm, Am) in path_states(x, b, h).items():
                if i < 0:
                    continue
                q = num(x["q"])[b, i, h]
                out, z, om, zm = M.T @ q, A.T @ q, Mm.T @ np.abs(q), Am.T @ np.abs(q)
                if cached:
                    nc = int(x["n_cache"][b])
                    g = gates_of(x, b, h, i) if gates_in is None else num(gates_in)[b, i, h]
                    gates[b, i, h, :nc] = g[:nc]
                    for j in reversed(range(nc)):
                        if not g[j] >= tau:
                            continue
                        At, Bc = num(x["At_cache"])[b, h, j], num(x["Bc_cache"])[b, h, j]
                        out, om = out + g[j] * (Bc.T @ z), om + g[j] * (np.abs(Bc).T @ zm)
                        z, zm = z + g[j] * (At.T @ z - z), zm + g[j] * (np.abs(At).T @ zm + zm)
                o[0, b, i, h], o[1, b, i, h] = out, om
    return o, gates


def call(x, **kw):
    d = {n: t.cuda() for n, t in x.items()}
    native = kw.pop("native", False)
    rest = {} if native else {m: d[m] for m in ("At_cur", "At_cache", "Bc_cache", "reps_cache", "n_cache")}
    if "gates_in" in kw:
        rest["reps_cache"] = None
    return hla.gdn_tree_decode(d["q"], d["k"], d["v"], d["beta"], d["alpha"], d["parent"], d["S_cur"], **rest, **kw)


def check(got, ref, terms, what):
    err, lim = np.abs(num(got.cpu()) - ref[0]), (6.0 * np.sqrt(terms / 3.0) + 24.0) * U * ref[1] + 1e-37
    assert (err <= lim).all(), f"{what}: {np.max(err / lim):.2f} of the bound at {np.argwhere(~(err <= lim))[0]}"
    return float(np.max(err / lim, initial=0.0))


CASES = [(1, 1, 1, 64, 64, "f32", 1, 1, "tree"), (2, 5, 2, 128, 128, "bf16", 3, 2, "tree"),
         (3, 16, 1, 64, 128, "bf16", 4, 33, "tree"), (2, 17, 2, 128, 64, "bf16", 2, 64, "chain"),
         (2, 32, 1, 128, 128, "bf16", 5, 5, "star"), (2, 33, 1, 128, 128, "bf16", 3, 7, "tree"),
         (1, 64, 1, 128, 128, "bf16", 2, 40, "chain"), (2, 64, 1, 64, 64, "bf16", 3, 1, "tree"),
         (1, 64, 1, 128, 64, "bf16", 2, 3, "tree"), (2, 64, 1, 64, 128, "f32", 2, 9, "tree"),
         (2, 7, 2, 128, 128, "f32", 3, 2, "tree"), (1, 20, 1, 128, 64, "f32", 9, 65, "chain"),
         (1, 64, 1, 128, 128, "f32", 3, 4, "star"), (1, 64, 1, 128, 64, "f32", 2, 4, "tree"),
         (2, 9, 2, 64, 64, "f32", 40, 3, "tree")]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_every_node_is_the_decode_step_after_its_ancestors(case):
    Bs, n, H, dk, dv, dtype, n_cap, n_rep, shape = case
    note(f"gdn_tree_decode {case}")
    x = make(Bs, n, H, dk, dv, dtype, n_cap, n_rep, shape=shape)
    terms = n + dk + n_cap * dk
    gates = torch.full((Bs, n, H, n_cap), 7.0, device="cuda")
    o = call(x, tau=0.3, gates_out=gates)
    ref, rg = reference(x, 0.3)
    # a gate that lies on the threshold would make two right answers
    assert not (np.abs(rg - 0.3) < 1e-5).any()
    w = check(o, ref, terms, "o")
    gerr = np.abs(num(gates.cpu()) - rg)
    # a score is a sum of dk products, the logit one of n_rep exponentials: relative to a gate below 1
    smax = np.abs(num(x["reps_cache"])).max() * np.abs(num(x["q"])).max() * np.sqrt(dk)
    assert gerr.max(initial=0.0) <= (6 * np.sqrt((dk + n_rep) / 3) + 24) * U * max(1.0, smax), gerr.max()
    nat = call(x, native=True)
    y = {k: v for k, v in x.items() if k not in ("At_cache",)}
    check(nat, reference(y, 0.3)[0], n + dk, "native o")
    note(f"  share of the bound: {w:.3f}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_given_gates_and_what_no_node_reads(dtype):
    note(f"gdn_tree_decode given gates {dtype}")
    x = make(2, 12, 2, 64, 128, dtype, 6, 2, seed=3)
    r = np.random.default_rng(5)
    g = torch.from_numpy(np.where(r.random((2, 12, 2, 6)) < 0.4, 0.2 + 0.8 * r.random((2, 12, 2, 6)), 0.05).astype(np.float32))
    g[:, :, :, 2] = 0.0          # no node reads chunk 2
    g[:, 5, :, 3] = float("nan")  # below every threshold
    x["At_cache"][:, :, 2] = float("nan")
    x["Bc_cache"][:, :, 2] = float("inf")
    o = call(x, tau=0.1, gates_in=g.cuda())
    ref = reference(x, 0.1, g)[0]
    check(o, ref, 12 + 64 + 6 * 64, "o")
    # a negative threshold lets every gate through but NaN; here none is left out by tau
    o2 = call(x, tau=2.0, gates_in=g.cuda())
    y = {k: v for k, v in x.items() if k != "At_cache"}
    check(o2, reference(y, 0.1)[0], 12 + 64, "o with every chunk below the threshold")


def test_absent_nodes():
    note("gdn_tree_decode absent nodes")
    x = make(2, 10, 2, 128, 64, "bf16", 3, 2, seed=4)
    x["parent"][0] = torch.tensor([-1, 0, 7, 2, -5, 4, 1, 6, 99, 8], dtype=torch.int32)
    x["parent"][1] = -2
    absent = {(0, i) for i in (2, 3, 4, 5, 8, 9)} | {(1, i) for i in range(10)}
    for name in ("q", "k", "v", "beta", "alpha"):
        for b, i in absent:
            x[name][b, i] = float("nan")
    gates = torch.full((2, 10, 2, 3), 7.0, device="cuda")
    o = call(x, tau=0.0, gates_out=gates)
    clean = {k: v.clone() for k, v in x.items()}
    for name in ("q", "k", "v", "beta", "alpha"):
        clean[name] = torch.nan_to_num(clean[name])
    check(o, reference(clean, 0.0)[0], 10 + 128 + 3 * 128, "o")
    for b, i in absent:
        assert (o[b, i] == 0).all() and (gates[b, i] == 0).all()


@pytest.mark.parametrize("case", [(1, 1, 1, 64, 64, "f32"), (4, 16, 2, 128, 128, "bf16"), (3, 64, 1, 64, 128, "bf16"),
                                  (3, 33, 2, 128, 64, "f32")], ids=str)
def test_accept(case):
    Bs, n, H, dk, dv, dtype = case
    note(f"gdn_tree_accept {case}")
    x = make(Bs, n, H, dk, dv, dtype, 3, 1, seed=6)
    node = np.array([n - 1, -1, n // 2, n + 3][:Bs], np.int32)
    commit = np.array([1, 1, 0, 1][:Bs], np.int32)
    x["n_cache"] = torch.tensor([1, 3, 2, 0][:Bs], dtype=torch.int32)
    want = {m: num(x[m]).copy() for m in ("S_cur", "At_cur", "At_cache", "Bc_cache", "n_cache")}
    mags = {m: np.zeros_like(want[m]) for m in ("S_cur", "At_cur", "At_cache", "Bc_cache")}
    for b in range(Bs):
        for h in range(H):
            at = path_states(x, b, h)
            M, A, Mm, Am = at[int(node[b])] if int(node[b]) in at else at[-1]
            want["S_cur"][b, h], want["At_cur"][b, h], mags["S_cur"][b, h], mags["At_cur"][b, h] = M, A, Mm, Am
            c = int(x["n_cache"][b])
            if commit[b] and c < 3:
                for live, cache, fresh in (("S_cur", "Bc_cache", 0.0), ("At_cur", "At_cache", np.eye(dk))):
                    want[cache][b, h, c], mags[cache][b, h, c] = want[live][b, h], mags[live][b, h]
                    want[live][b, h], mags[live][b, h] = fresh, 0.0
        if commit[b] and want["n_cache"][b] < 3:
            want["n_cache"][b] += 1
    d = {m: t.cuda() for m, t in x.items()}
    hla.gdn_tree_accept(d["k"], d["v"], d["beta"], d["alpha"], d["parent"], torch.from_numpy(node).cuda(), d["S_cur"],
                        At_cur=d["At_cur"], At_cache=d["At_cache"], Bc_cache=d["Bc_cache"], n_cache=d["n_cache"],
                        commit=torch.from_numpy(commit).cuda())
    torch.cuda.synchronize()
    assert np.array_equal(d["n_cache"].cpu().numpy(), want["n_cache"])
    for m, mag in mags.items():
        lim = (6 * np.sqrt((n + dk) / 3) + 24) * U * mag
        if m.endswith("cache") and dtype == "bf16":
            lim = lim + 2.0 ** -8 * np.abs(want[m]) * (mag > 0)
        assert (np.abs(num(d[m].cpu()) - want[m]) <= lim).all(), m
    # the state alone, without a transition
    S = x["S_cur"].cuda()
    hla.gdn_tree_accept(d["k"], d["v"], d["beta"], d["alpha"], d["parent"], torch.from_numpy(node).cuda(), S)
    b = 2 if Bs > 2 else 0
    if not commit[b]:
        assert torch.equal(S[b], d["S_cur"][b])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_draft_verify_accept_is_decoding_token_by_token(dtype):
    """A run of drafted trees, each with one accepted path, against gdn_decode on the accepted tokens:
    the live chunk is committed in between, on both sides."""
    note(f"draft, verify, accept {dtype}")
    Bs, n, H, dk, dv, n_cap, n_rep = 2, 6, 2, 128, 64, 4, 3
    x = make(Bs, n, H, dk, dv, dtype, n_cap, n_rep, seed=8)
    d = {m: t.cuda() for m, t in x.items()}
    d["n_cache"] = torch.tensor([1, 2], dtype=torch.int32, device="cuda")
    a = {m: d[m].clone() for m in ("S_cur", "At_cur", "At_cache", "Bc_cache", "n_cache")}
    e = {m: d[m].clone() for m in ("S_cur", "At_cur", "At_cache", "Bc_cache", "n_cache")}
    tol = (6 * np.sqrt((n + dk + n_cap * dk) / 3) + 24) * U
    for step in range(3):
        t = {m: v.cuda() for m, v in make(Bs, n, H, dk, dv, dtype, 0, 0, seed=20 + step).items()}
        t["parent"] = torch.tensor([[-1, 0, 0, 2, 3, 1]] * Bs, dtype=torch.int32, device="cuda")
        path, node = [0, 2, 3], torch.full((Bs,), 3, dtype=torch.int32, device="cuda")
        commit = torch.full((Bs,), int(step == 1), dtype=torch.int32, device="cuda")
        o = hla.gdn_tree_decode(t["q"], t["k"], t["v"], t["beta"], t["alpha"], t["parent"], a["S_cur"], At_cur=a["At_cur"],
                                At_cache=a["At_cache"], Bc_cache=a["Bc_cache"], reps_cache=d["reps_cache"],
                                n_cache=a["n_cache"], tau=0.3)
        hla.gdn_tree_accept(t["k"], t["v"], t["beta"], t["alpha"], t["parent"], node, **a, commit=commit)
        for i in path:
            tok = [t[m][:, i].contiguous() for m in ("q", "k", "v", "beta", "alpha")]
            oi = hla.gdn_decode(*tok, e["S_cur"], At_cur=e["At_cur"], At_cache=e["At_cache"], Bc_cache=e["Bc_cache"],
                                reps_cache=d["reps_cache"], n_cache=e["n_cache"], tau=0.3,
                                commit=bool(step == 1 and i == path[-1]))
            # both are within the bound of the same value; magnitudes grow by a factor below 8 here
            assert (o[:, i] - oi).abs().max() <= 16 * tol * oi.abs().max()
        assert torch.equal(a["n_cache"], e["n_cache"])
        for m in ("S_cur", "At_cur"):
            assert (a[m] - e[m]).abs().max() <= 16 * tol * max(1.0, e[m].abs().max())
