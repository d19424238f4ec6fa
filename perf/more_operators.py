"""Timed cases of linear attention with a decay for each head, and of trees of drafted tokens.

Linear attention with a decay keeps, per head, a state M [dk, dv] and does for each token

    M_t = exp(g_t) M_{t-1} + k_t v_t^T,        o_t = M_t^T q_t

with g_t <= 0 (-inf clears the state), given per token or one number for each head.  A prompt runs
in chunks, a single token updates the state in place, and training also needs the gradients.
Query and key heads may be shared by groups of value heads; rows of a padded batch have lengths.

A tree of drafted tokens continues the state of a gated delta rule decode: each token does

    M_i = alpha_i (I - beta_i k_i k_i^T) M_p + beta_i k_i v_i^T,    p the parent of i

from its parent's state (the live state for a parent of -1), and reads the cached chunk maps with
gates of its own, newest chunk first.  Afterwards the accepted path enters the live state.

``run`` computes each operator in elementary torch operations, or, where ``own`` is true, through
the library.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
C = 64  # tokens per chunk of the plain chunked form
CLEAR = -1.0e4  # exp() of this is zero: stands for a logarithm of -inf


# ------------------------------------------------------------------------------- cases
def _la(name, op, B, T, H, Hk, dk, dv, dtype, per_head=False, ragged=False, start=False):
    return dict(name=name, op=op, B=B, T=T, H=H, Hk=Hk, dk=dk, dv=dv, dtype=dtype, per_head=per_head, ragged=ragged,
                start=start)


def _tree(name, op, Bs, H, n, dk, dv, dtype, chunks, n_rep, ragged=False, active=0.0, commit=False):
    return dict(name=name, op=op, Bs=Bs, H=H, n=n, dk=dk, dv=dv, dtype=dtype, chunks=chunks, n_rep=n_rep,
                ragged=ragged, active=active, commit=commit)


def listed():
    return [
        # the prompt of a short question: latency
        _la("prompt_short", "prefill", 1, 37, 16, 16, 128, 128, "bf16"),
        # one document of 65536 tokens that continues a state: few heads, long
        _la("prompt_long", "prefill", 1, 65536, 16, 16, 128, 128, "bf16", start=True),
        # a padded batch, lengths from none to all, query and key heads shared, one decay a head, float32
        _la("prompt_padded", "prefill", 13, 1531, 12, 4, 64, 128, "f32", per_head=True, ragged=True),
        # single tokens: one conversation, and a full serving batch
        _la("step_one", "step", 1, 1, 16, 16, 128, 128, "bf16"),
        _la("step_batch", "step", 256, 1, 16, 4, 128, 128, "bf16"),
        # training: a batch of four sequences of 4096 tokens
        _la("train_batch", "train", 4, 4096, 16, 16, 128, 128, "bf16"),
        # training in float32 on a padded batch, shared heads, one learned decay a head, from a given state
        _la("train_padded", "train", 5, 1000, 12, 3, 128, 64, "f32", per_head=True, ragged=True, start=True),
        # drafted tokens of one conversation, eight cached chunks
        _tree("tree_one", "tree", 1, 16, 7, 128, 128, "bf16", 8, 2),
        # a serving batch, sixteen drafted tokens each, 64 chunks scored by their own keys
        _tree("tree_batch", "tree", 64, 16, 16, 128, 128, "bf16", 64, 64),
        # requests of every length and trees of every size, the caller's gates, float32 maps
        _tree("tree_mixed", "tree", 21, 5, 33, 64, 128, "f32", 100, 3, ragged=True, active=0.25),
        # the accepted tokens of one conversation, and of a batch in which some live chunks are complete
        _tree("accept_one", "accept", 1, 16, 7, 128, 128, "bf16", 1, 0),
        _tree("accept_batch", "accept", 64, 16, 16, 128, 128, "bf16", 4, 0, ragged=True, commit=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "train", "train", "step", "tree", "tree", "accept"])
    dk, dv, dtype = rng.choice([64, 128]), rng.choice([64, 128]), rng.choice(["bf16", "bf16", "f32"])
    if op in ("prefill", "train", "step"):
        H = rng.choice([1, 2, 3, 4, 6, 8, 12, 16])
        Hk = H // rng.choice([d for d in (1, 1, 2, 3, 4) if H % d == 0])
        most = {"prefill": 1 << 20, "train": 1 << 17, "step": 4096}[op]
        T = 1 if op == "step" else _log_int(rng, 1, 65536 if op == "prefill" else 8192)
        B = _log_int(rng, 1, max(1, min(4096, most // (T * H))))
        case = _la("", op, B, T, H, Hk, dk, dv, dtype, rng.random() < 0.3, op != "step" and rng.random() < 0.4,
                   rng.random() < 0.5)
    else:
        H, n = rng.choice([1, 2, 3, 5, 8, 16]), _log_int(rng, 1, 64)
        if op == "tree":
            chunks = _log_int(rng, 1, 1024)
            rows = _log_int(rng, 1, max(1, min(1024, 32768 // (chunks * max(1, n // 16)))))
            case = _tree("", op, max(1, rows // H), H, n, dk, dv, dtype, chunks, _log_int(rng, 1, 64),
                         rng.random() < 0.5, rng.choice([0.0, 0.0, 0.25, 0.6]))
        else:
            case = _tree("", op, max(1, _log_int(rng, 1, 1024) // H), H, n, dk, dv, dtype, rng.randint(1, 6), 0,
                         rng.random() < 0.5, 0.0, rng.random() < 0.5)
    case.pop("name")
    return case


def _tokens(case):
    """Tokens of all rows that count: about half where lengths are mixed."""
    return case["B"] * case["T"] * (0.5 if case["ragged"] and case["B"] > 1 else 1.0)


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    H, dk, dv = case["H"], case["dk"], case["dv"]
    if case["op"] in ("prefill", "train", "step"):
        Hk, B, n = case["Hk"], case["B"], _tokens(case)
        token = e * (2 * Hk * dk + 2 * H * dv) + (0 if case["per_head"] else 4 * H)
        state = 4 * B * H * dk * dv
        flops = n * H * 4 * dk * dv
        if case["op"] == "step":
            return {"bytes": float(2 * state + n * token), "flops": float(flops)}
        states = state * (2 if case["start"] else 1)
        if case["op"] == "prefill":
            return {"bytes": float(states + n * token), "flops": float(flops)}
        # the forward call, then q, k, v, dO and the final state's gradient to those of all inputs
        back = n * (e * (4 * Hk * dk + 3 * H * dv) + (0 if case["per_head"] else 8 * H)) + 3 * state
        return {"bytes": float(states + n * token + back), "flops": float(flops + 3.5 * flops)}
    rows, n = case["Bs"] * H, case["n"] * (0.5 if case["ragged"] else 1.0)
    maps, live = dk * (dk + dv), 4 * dk * (dk + dv)
    token = (2 * dk + dv) * e + 8
    if case["op"] == "accept":
        made = rows * maps * e * (0.25 if case["commit"] else 0.0)
        return {"bytes": float(2 * rows * live + rows * n * token * 0.5 + made), "flops": float(rows * n * 2 * maps)}
    held = rows * case["chunks"] * (0.5 if case["ragged"] else 1.0)
    # of drafted tokens that each read a part of the chunks, some token reads nearly every chunk
    some = 1.0 - (1.0 - case["active"]) ** case["n"] if case["active"] else 1.0
    scored = 0.0 if case["active"] else held * case["n_rep"] * dk
    nbytes = (held * some * maps + scored) * e + rows * (live + n * (token + 4 * dv))
    if case["active"]:
        nbytes += 4 * n * held
    nbytes += 4 * n * held  # the gates are returned
    share = case["active"] or 1.0
    return {"bytes": float(nbytes), "flops": float(2 * n * (held * share * maps + scored + rows * maps))}


# ------------------------------------------------------------------------------ inputs
def _unit(x):
    return torch.nn.functional.normalize(x, dim=-1)


def _prepare_la(case, gen, rand, randn):
    B, T, H, Hk, dk, dv = (case[x] for x in ("B", "T", "H", "Hk", "dk", "dv"))
    dtype = TYPES[case["dtype"]]
    lead = (B,) if case["op"] == "step" else (B, T)
    s = dict(case=case)
    s["q"], s["k"] = (_unit(randn(*lead, Hk, dk)).to(dtype) for _ in range(2))
    s["v"] = randn(*lead, H, dv).to(dtype)
    if case["per_head"]:  # decays spread over the heads, about 1 in 16 to 1 in 1000 a token
        s["g"] = -torch.exp2(-4.0 - 6.0 * rand(H))
    else:  # slow decays that depend on the token; now and then a new document clears the state
        s["g"] = -torch.nn.functional.softplus(randn(*lead, H) - 3.0)
        if case["op"] != "step":
            s["g"][rand(*lead, H) < 1e-3] = -math.inf
    if case["op"] == "step":
        s["S"] = 0.3 * randn(B, H, dk, dv)
        return s
    if case["ragged"]:  # every length from none to all
        n = torch.linspace(T, 0, B, device="cuda").round().to(torch.int32)
        s["lens"] = n[torch.randperm(B, generator=gen, device="cuda")]
    if case["start"]:
        s["S0"] = 0.3 * randn(B, H, dk, dv)
    if case["op"] == "train":
        s["dO"] = randn(B, T, H, dv).to(dtype)
        s["dS"] = 0.3 * randn(B, H, dk, dv)
    return s


def _chunk_bank(count, dk, dv, gen):
    """Maps of `count` chunks of 64 tokens: M -> At M + Bc."""
    k = _unit(torch.randn(count, C, dk, generator=gen, device="cuda"))
    v = torch.randn(count, C, dv, generator=gen, device="cuda")
    beta = 0.02 + 0.18 * torch.rand(count, C, 1, 1, generator=gen, device="cuda")
    alpha = 0.997 + 0.003 * torch.rand(count, C, 1, 1, generator=gen, device="cuda")
    At = torch.eye(dk, device="cuda").repeat(count, 1, 1)
    Bc = torch.zeros(count, dk, dv, device="cuda")
    for t in range(C):
        kt, vt = k[:, t, :, None], v[:, t, None, :]
        At = alpha[:, t] * (At - beta[:, t] * kt * (kt * At).sum(-2, keepdim=True))
        Bc = alpha[:, t] * (Bc - beta[:, t] * kt * (kt * Bc).sum(-2, keepdim=True)) + beta[:, t] * kt * vt
    return At, Bc


def _prepare_tree(case, gen, rand, randn):
    Bs, H, n, dk, dv, chunks, n_rep = (case[x] for x in ("Bs", "H", "n", "dk", "dv", "chunks", "n_rep"))
    dtype = TYPES[case["dtype"]]
    s = dict(case=case)
    common = randn(Bs, 1, H, dk)  # the drafted tokens' queries look for similar things
    s["q"] = (0.9 * common + 0.4 * randn(Bs, n, H, dk)).to(dtype)
    s["k"] = _unit(randn(Bs, n, H, dk)).to(dtype)
    s["v"] = randn(Bs, n, H, dv).to(dtype)
    s["beta"], s["alpha"] = rand(Bs, n, H), 0.8 + 0.2 * rand(Bs, n, H)
    # runs of tokens with side branches; a shorter tree's places at the end hold no token (-2)
    i = torch.arange(n, device="cuda").expand(Bs, n)
    back = torch.where(rand(Bs, n) < 0.6, 1, 1 + (rand(Bs, n) * 6).long())
    parent = (i - back).clamp(min=-1)
    if case["ragged"]:
        size = 1 + (rand(Bs, 1) * n).long()
        parent = torch.where(i < size, parent, -2)
    s["parent"] = parent.to(torch.int32)
    s["S_cur"] = 0.1 * randn(Bs, H, dk, dv)
    s["At_cur"] = torch.eye(dk, device="cuda") - 0.02 * rand(Bs, H, dk, dk)
    A, B = _chunk_bank(48, dk, dv, gen)
    if case["op"] == "accept":
        pick = torch.randint(0, 48, (Bs * H * chunks,), generator=gen, device="cuda")
        node = (rand(Bs) * (parent >= -1).sum(-1)).long()
        s["node"] = torch.where(rand(Bs) < 0.1, -1, node).to(torch.int32)
        if case["commit"]:
            s["commit"] = (rand(Bs) < 0.25).to(torch.int32)
            s["n_cache"] = (rand(Bs) * (chunks + 1)).to(torch.int32)
            s["At_cache"] = A.to(dtype)[pick].view(Bs, H, chunks, dk, dk)
            s["Bc_cache"] = B.to(dtype)[pick].view(Bs, H, chunks, dk, dv)
        return s
    pick = torch.randint(0, 48, (Bs * H * chunks,), generator=gen, device="cuda")
    s["At_cache"] = A.to(dtype)[pick].view(Bs, H, chunks, dk, dk)
    s["Bc_cache"] = B.to(dtype)[pick].view(Bs, H, chunks, dk, dv)
    s["n_cache"] = torch.full((Bs,), chunks, dtype=torch.int32, device="cuda")
    if case["ragged"]:
        s["n_cache"] = torch.linspace(chunks, 0, Bs, device="cuda").round().to(torch.int32)
    s["tau"] = 1e-3
    if case["active"]:
        s["tau"] = 0.1
        on = rand(Bs, n, H, chunks) < case["active"]
        s["gates_in"] = torch.where(on, 0.15 + 0.8 * rand(Bs, n, H, chunks), 0.08 * rand(Bs, n, H, chunks))
    else:  # keys of a chunk whose logit lies near a level of its own between -5 and -1
        s["reps"] = torch.empty(Bs, H, chunks, n_rep, dk, dtype=dtype, device="cuda")
        for b in range(Bs):
            c = common[b, 0]
            level = -5.0 + 4.0 * rand(H, chunks, 1, 1)
            s["reps"][b] = 0.3 * randn(H, chunks, n_rep, dk) + level * (
                math.sqrt(dk) * c / c.square().sum(-1, keepdim=True))[:, None, None, :]
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *shape: torch.rand(shape, generator=gen, device="cuda")  # noqa: E731
    randn = lambda *shape: torch.randn(shape, generator=gen, device="cuda")  # noqa: E731
    make = _prepare_la if case["op"] in ("prefill", "train", "step") else _prepare_tree
    return make(case, gen, rand, randn)


# -------------------------------------------------------- plain forms: linear attention
def _decays(lg):
    """exp(lg_i - lg_j) for j <= i, else 0, of sums lg [..., n] in 64 bits."""
    n = lg.shape[-1]
    i = torch.arange(n, device=lg.device)
    diff = (lg[..., :, None] - lg[..., None, :]).masked_fill(i[:, None] < i, -math.inf)
    return diff.exp().float()


def _plain_forward(q, k, v, g, S0, lens):
    """The chunked form in 32 bits; sums of logarithms in 64.  q, k [B,T,Hk,dk], v [B,T,H,dv]."""
    B, T, H, dv = v.shape
    dk, N = k.shape[-1], -(-T // C)
    here = torch.ones(B, T, dtype=torch.bool, device=v.device)
    if lens is not None:
        here = torch.arange(T, device=v.device) < lens[:, None]
    wide = here[:, :, None, None]
    g = g.double().clamp(min=CLEAR).expand(B, T, H) * here[:, :, None]
    group = H // k.shape[2]
    q, k = (torch.where(wide, x, 0.0).repeat_interleave(group, 2) for x in (q, k))
    v = torch.where(wide, v, 0.0)
    pad = N * C - T

    def chunks(x):  # [B, H, N, C, ...]
        x = torch.nn.functional.pad(x, (0, 0) * (x.dim() - 2) + (0, pad))
        return x.view(B, N, C, *x.shape[2:]).movedim(3, 1)

    q, k, v, g = (chunks(x) for x in (q, k, v, g))
    lg = g.cumsum(-1)
    o = torch.matmul(torch.matmul(q, k.mT) * _decays(lg), v)
    gain = torch.matmul((k * (lg[..., -1:] - lg).exp().float()[..., None]).mT, v)  # what each chunk adds
    total = lg[..., -1].cumsum(-1)
    start = torch.nn.functional.pad(total, (1, 0))  # the decay up to each boundary
    keep = _decays(start)[..., 1:]  # of chunk m's gain at boundary n: from boundary m + 1 on
    M = torch.matmul(keep, gain.flatten(-2)).view(B, H, N + 1, dk, dv)
    if S0 is not None:
        M = M + start.exp().float()[..., None, None] * S0[:, :, None]
    o = o + torch.matmul(q * lg.exp().float()[..., None], M[:, :, :-1])
    o = o.movedim(1, 3).reshape(B, N * C, H, dv)[:, :T]
    return torch.where(wide, o, 0.0), M[:, :, -1]


def _plain_prefill(s):
    o, S = _plain_forward(s["q"].float(), s["k"].float(), s["v"].float(), s["g"], s.get("S0"), s.get("lens"))
    return dict(o=o.to(s["q"].dtype), S_final=S)


def _plain_train(s):
    dtype = s["q"].dtype
    ins = [s[x].float().detach().requires_grad_(True) for x in ("q", "k", "v", "g")]
    if "S0" in s:
        ins.append(s["S0"].detach().requires_grad_(True))
    o, S = _plain_forward(*ins[:4], ins[4] if "S0" in s else None, s.get("lens"))
    d = torch.autograd.grad([o, S], ins, [s["dO"].float(), s["dS"]])
    out = dict(o=o.detach().to(dtype), S_final=S.detach(), dq=d[0].to(dtype), dk=d[1].to(dtype), dv=d[2].to(dtype),
               dg=d[3])
    if "S0" in s:
        out["dS0"] = d[4]
    return out


def _plain_step(s):
    group = s["case"]["H"] // s["case"]["Hk"]
    q, k = (s[x].float().repeat_interleave(group, 1) for x in ("q", "k"))
    S = s["S"]
    S.mul_(s["g"].exp().expand(S.shape[:2])[..., None, None]).add_(k[..., None] * s["v"].float()[..., None, :])
    return dict(o=(q[..., None] * S).sum(-2).to(s["q"].dtype), S=S)


# ---------------------------------------------------------- plain forms: drafted tokens
def _doubled(P):
    """(I - P)^-1 of a nilpotent P: the product of I + P^(2^i)."""
    n = P.shape[-1]
    eye = torch.eye(n, dtype=P.dtype, device=P.device)
    out = eye + P
    for _ in range(max(0, n - 1).bit_length()):
        P = torch.matmul(P, P)
        out = out + torch.matmul(out, P)
    return out


def _solve(s):
    """The tree's closed form, per head: (D, gamma, U, W, k) with D_ij the decay from ancestor j to i
    (0 where j is none; 1 at i), gamma the decay from the live state, and U, W solving
    u_j = beta_j (v_j - what the ancestors' u hold at k_j), W the same for the live state."""
    n = s["case"]["n"]
    parent = s["parent"].long()
    i = torch.arange(n, device=parent.device)
    fine = (parent >= -1) & (parent < i)
    P = ((parent[:, :, None] == i) & fine[:, :, None]).double()
    anc = _doubled(P)  # ancestors and itself
    fine = torch.matmul(anc, (~fine).double()[..., None])[..., 0] == 0
    anc = (anc * fine[:, :, None])[:, None]
    k, v = (s[x].float().transpose(1, 2) for x in ("k", "v"))
    beta = s["beta"].transpose(1, 2).double()
    lg = torch.matmul(anc, s["alpha"].transpose(1, 2).double().log()[..., None])[..., 0]
    D = torch.where(anc > 0, (lg[..., :, None] - lg[..., None, :]).exp(), 0.0)
    gamma = lg.exp() * fine[:, None]
    L = beta[..., None] * D * torch.matmul(k, k.mT).double()
    L = L * (i[:, None] != i)
    X = _doubled(-L) * beta[..., None, :]
    U = torch.matmul(X.float(), v)
    W = torch.matmul((X * gamma[..., None, :]).float(), k)
    return D.float(), gamma.float(), U, W, k


def _plain_tree(s):
    case, tau = s["case"], s["tau"]
    D, gamma, U, W, k = _solve(s)
    q = s["q"].float().transpose(1, 2)
    P = D * torch.matmul(q, k.mT)
    r = gamma[..., None] * q - torch.matmul(P, W)
    o = torch.matmul(P, U) + torch.matmul(r, s["S_cur"])
    z = torch.matmul(r, s["At_cur"])
    scale = 1.0 / math.sqrt(case["dk"])
    there = torch.diagonal(D, dim1=-2, dim2=-1) > 0
    gates = torch.empty(*s["parent"].shape, case["H"], case["chunks"], device=q.device)
    # each chunk acts on what the newer ones left: the recursion over the chunks, newest first
    for j in reversed(range(case["chunks"])):
        if "gates_in" in s:
            g = s["gates_in"][..., j].transpose(1, 2)
        else:
            score = torch.matmul(q, s["reps"][:, :, j].float().mT) * scale
            top = score.amax(-1, keepdim=True)
            logit = top[..., 0] + (score - top).exp().mean(-1).log()
            g = 1.0 / (1.0 + (-logit).exp())
        g = torch.where((j < s["n_cache"])[:, None, None] & there, g, 0.0)
        gates[..., j] = g.transpose(1, 2)
        g = torch.where(g >= tau, g, 0.0)[..., None]
        o = o + g * torch.matmul(z, s["Bc_cache"][:, :, j].float())
        z = z + g * (torch.matmul(z, s["At_cache"][:, :, j].float()) - z)
    return dict(o=o.transpose(1, 2).contiguous(), gates=gates)


def _plain_accept(s):
    case = s["case"]
    Bs, H, n, chunks = (case[x] for x in ("Bs", "H", "n", "chunks"))
    D, gamma, U, W, k = _solve(s)
    M, At = s["S_cur"], s["At_cur"]
    node = s["node"].long()
    b = torch.arange(Bs, device=node.device)
    at = node.clamp(0, n - 1)
    on = ((node >= 0) & (node < n))[:, None] & (D[b, :, at, at] > 0)  # the node is there
    on = on[..., None, None]
    path = D[b, :, at][..., None] * k  # [Bs, H, n, dk]: each ancestor's key, decayed to the node
    ga = gamma[b, :, at][..., None, None]
    # from the node's closed form: M = gamma M_0 + sum_j D_j k_j (u_j - M_0^T w_j)^T
    newM = ga * M + torch.matmul(path.mT, U - torch.matmul(W, M))
    newA = ga * At - torch.matmul(path.mT, torch.matmul(W, At))
    M.copy_(torch.where(on, newM, M))
    At.copy_(torch.where(on, newA, At))
    if not case["commit"]:
        return dict(S_cur=M, At_cur=At)
    count = s["n_cache"].clone()  # the cache takes the same chunks in every pass
    made = (s["commit"] != 0) & (count >= 0) & (count < chunks)
    slot = count.clamp(0, chunks - 1).long()
    wide = made[:, None, None, None]
    for cache, live, fresh in (("At_cache", At, torch.eye(case["dk"], device="cuda")), ("Bc_cache", M, 0.0 * M[:1, :1])):
        c = s[cache]
        c[b, :, slot] = torch.where(wide, live.to(c.dtype), c[b, :, slot])
        live.copy_(torch.where(wide, fresh, live))
    count += made.to(torch.int32)
    return dict(S_cur=M, At_cur=At, At_cache=s["At_cache"], Bc_cache=s["Bc_cache"], n_cache=count)


def run(s):
    if own:
        return _own(s)
    plain = dict(prefill=_plain_prefill, train=_plain_train, step=_plain_step, tree=_plain_tree, accept=_plain_accept)
    return plain[s["case"]["op"]](s)


# ------------------------------------------------------------------------ the framework
def _own(s):
    from gated_deltanet_hybrid_amd import hla
    op = s["case"]["op"]
    if op == "step":
        return dict(o=hla.la_decode(s["q"], s["k"], s["v"], s["g"], s["S"]), S=s["S"])
    if op in ("prefill", "train"):
        args = (s["q"], s["k"], s["v"], s["g"])
        o, S = hla.la_prefill(*args, S0=s.get("S0"), lens=s.get("lens"))
        if op == "prefill":
            return dict(o=o, S_final=S)
        d = hla.la_prefill_backward(*args, s["dO"], dS_final=s["dS"], S0=s.get("S0"), lens=s.get("lens"),
                                    want_dS0="S0" in s)
        out = dict(o=o, S_final=S, dq=d["dq"], dk=d["dk"], dv=d["dv"], dg=d["dlog_decay"])
        if "S0" in s:
            out["dS0"] = d["dS0"]
        return out
    token = (s["k"], s["v"], s["beta"], s["alpha"], s["parent"])
    if op == "tree":
        gates = torch.empty(*s["parent"].shape, s["case"]["H"], s["case"]["chunks"], device="cuda")
        o = hla.gdn_tree_decode(s["q"], *token, s["S_cur"], At_cur=s["At_cur"], At_cache=s["At_cache"],
                                Bc_cache=s["Bc_cache"], reps_cache=s.get("reps"), n_cache=s["n_cache"],
                                gates_in=s.get("gates_in"), tau=s["tau"], gates_out=gates)
        return dict(o=o, gates=gates)
    if not s["case"]["commit"]:
        hla.gdn_tree_accept(*token, s["node"], s["S_cur"], At_cur=s["At_cur"])
        return dict(S_cur=s["S_cur"], At_cur=s["At_cur"])
    count = s["n_cache"].clone()  # the cache takes the same chunks in every pass
    hla.gdn_tree_accept(*token, s["node"], s["S_cur"], At_cur=s["At_cur"], At_cache=s["At_cache"],
                        Bc_cache=s["Bc_cache"], n_cache=count, commit=s["commit"])
    return dict(S_cur=s["S_cur"], At_cur=s["At_cur"], At_cache=s["At_cache"], Bc_cache=s["Bc_cache"], n_cache=count)


# ------------------------------------------------------------------ the definition, 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "tree":
        return _exact_tree(s)
    if case["op"] == "accept":
        return _exact_accept(s)
    if case["T"] > 20000 and case["op"] == "train":
        return None
    return _exact_la(s)


def _exact_la(s):
    """Token by token; the gradients by the reverse recurrence, states replayed in blocks."""
    case = s["case"]
    B, T, H, Hk, dk, dv = (case[x] for x in ("B", "T", "H", "Hk", "dk", "dv"))
    step = case["op"] == "step"
    head = torch.arange(H, device="cuda") // (H // Hk)
    grow = (lambda x: x.double()[:, None]) if step else (lambda x: x.double())
    q, k, v = (grow(s[x]) for x in ("q", "k", "v"))
    g = (s["g"].double() if case["per_head"] else grow(s["g"])).expand(B, T, H)
    here = torch.ones(B, T, dtype=torch.float64, device="cuda")
    if "lens" in s:
        here = (torch.arange(T, device="cuda") < s["lens"][:, None]).double()
    a = torch.where(here[..., None] > 0, g.exp(), 1.0)[..., None, None]
    on = here[:, :, None, None]
    M = s["S"].double().clone() if step else s["S0"].double().clone() if case["start"] else torch.zeros(
        B, H, dk, dv, dtype=torch.float64, device="cuda")
    kt = lambda t: (k[:, t] * on[:, t])[:, head]  # noqa: E731
    qt = lambda t: (q[:, t] * on[:, t])[:, head]  # noqa: E731
    update = lambda M, t: a[:, t] * M + kt(t)[..., None] * v[:, t, :, None]  # noqa: E731
    o = torch.zeros(B, T, H, dv, dtype=torch.float64, device="cuda")
    block, kept = 64, []
    for t in range(T):
        if t % block == 0:
            kept.append(M)
        M = update(M, t)
        o[:, t] = (qt(t)[..., None] * M).sum(-2)
    if step:
        return dict(o=o[:, 0], S=M)
    out = dict(o=o, S_final=M)
    if case["op"] == "prefill":
        return out
    G = s["dS"].double()
    dO = s["dO"].double()
    dq, dk_, dv_ = torch.zeros(B, T, H, dk, dtype=torch.float64, device="cuda"), torch.zeros(
        B, T, H, dk, dtype=torch.float64, device="cuda"), torch.zeros(B, T, H, dv, dtype=torch.float64, device="cuda")
    dg = torch.zeros(B, T, H, dtype=torch.float64, device="cuda")
    for first in reversed(range(0, T, block)):
        states = [kept[first // block]]
        last = min(T, first + block)
        for t in range(first, last):
            states.append(update(states[-1], t))
        for t in reversed(range(first, last)):
            do = dO[:, t] * on[:, t]
            G = G + qt(t)[..., None] * do[:, :, None]
            dq[:, t] = (states[t - first + 1] * do[:, :, None]).sum(-1)
            dk_[:, t] = (G * v[:, t, :, None]).sum(-1) * on[:, t]
            dv_[:, t] = (G * kt(t)[..., None]).sum(-2)
            dg[:, t] = (G * a[:, t] * states[t - first]).sum((-2, -1)) * here[:, t, None]
            G = a[:, t] * G
    shared = lambda x: x.view(B, T, Hk, H // Hk, dk).sum(3)  # noqa: E731
    out.update(dq=shared(dq), dk=shared(dk_), dv=dv_, dg=dg.sum((0, 1)) if case["per_head"] else dg)
    if case["start"]:
        out["dS0"] = G
    return out


def _path_states(s, live, b, write):
    """Every node's state of sequence b from `live` [H, dk, w], token by token, or None where it is absent."""
    n = s["case"]["n"]
    parent = s["parent"][b].tolist()
    k, v, beta, alpha = (s[x][b].double() for x in ("k", "v", "beta", "alpha"))
    at = {-1: live}
    for i in range(n):
        if parent[i] >= i or parent[i] not in at:
            continue
        M, kk, be = at[parent[i]], k[i][..., None], beta[i][:, None, None]
        M = alpha[i][:, None, None] * (M - be * kk * (kk * M).sum(-2, keepdim=True))
        at[i] = M + be * kk * v[i][:, None, :] if write else M
    return at


def _exact_tree(s):
    case = s["case"]
    Bs, H, n, dk, dv = (case[x] for x in ("Bs", "H", "n", "dk", "dv"))
    if Bs * n * (1 + case["chunks"] / 8) > 60000:
        return None
    out = torch.zeros(Bs, n, H, dv, dtype=torch.float64, device="cuda")
    gates = torch.zeros(Bs, n, H, case["chunks"], dtype=torch.float64, device="cuda")
    for b in range(Bs):
        states = _path_states(s, s["S_cur"][b].double(), b, True)
        maps = _path_states(s, s["At_cur"][b].double(), b, False)
        there = [i for i in range(n) if i in states]
        if not there:
            continue
        q = s["q"][b].double()[there]  # [m, H, dk]
        o = torch.stack([(q[x][..., None] * states[i]).sum(-2) for x, i in enumerate(there)])
        y = torch.stack([(q[x][..., None] * maps[i]).sum(-2) for x, i in enumerate(there)])
        held = int(s["n_cache"][b])
        if "gates_in" in s:
            g = s["gates_in"][b, there, :, :held].double()
        else:
            e = (torch.matmul(s["reps"][b, :, :held].double(), q.movedim(0, -1)[:, None]) / math.sqrt(dk)).exp().mean(2)
            g = (e / (1 + e)).movedim(-1, 0)  # [m, H, held]
        gates[b, there, :, :held] = g
        g = torch.where(g >= s["tau"], g, 0.0)
        # the states composed oldest first, M -> M + g (At M + Bc - M), then read with y: the definition
        past = torch.zeros(len(there), H, dk, dv, dtype=torch.float64, device="cuda")
        for j in range(held):
            move = torch.matmul(s["At_cache"][b, :, j].double(), past) + s["Bc_cache"][b, :, j].double() - past
            past = past + g[:, :, j, None, None] * move
        out[b, there] = o + (y[..., None] * past).sum(-2)
    return dict(o=out, gates=gates)


def _exact_accept(s):
    case = s["case"]
    out = dict(S_cur=s["S_cur"].double(), At_cur=s["At_cur"].double())
    for b, node in enumerate(s["node"].tolist()):
        for name, write in (("S_cur", True), ("At_cur", False)):
            at = _path_states(s, out[name][b].clone(), b, write)
            out[name][b] = at[node] if node >= 0 and node in at else at[-1]
    if not case["commit"]:
        return out
    out.update(At_cache=s["At_cache"].double(), Bc_cache=s["Bc_cache"].double(), n_cache=None)
    for b, (c, held) in enumerate(zip(s["commit"].tolist(), s["n_cache"].tolist())):
        if c and held < case["chunks"]:
            for name, cache, fresh in (("S_cur", "Bc_cache", 0.0), ("At_cur", "At_cache", torch.eye(
                    case["dk"], dtype=torch.float64, device="cuda"))):
                out[cache][b, :, held] = out[name][b]
                out[name][b] = fresh
    return out
