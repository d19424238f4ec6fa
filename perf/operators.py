"""Timed cases of the 8-bit chunk cache: filling it, decoding over it, evicting from it.

A decoding program keeps, per sequence and head, the affine maps of the prefix's chunks
(S -> S A + B) and a few representative keys of each chunk, in 8 bits with one scale per chunk
and head for A - I, for B and for the keys.  A decode step scores the chunks by their keys,
composes the chunks whose gate reaches tau and adds every gate to its chunk's weight; when the
cache is full the chunks of least weight leave it.

``run`` computes each operator in elementary torch operations, or, where ``own`` is true, through
the library.  Every cache is a dict of

    maps   [Bs, H, n_cap, dk + dv, dk]   8 bits: rows of A - I, then rows of B (S is [dv, dk])
    reps   [Bs, H, n_cap, n_rep, dk]     8 bits
    scale  [Bs, H, n_cap, 4]             float32: of A - I, of B, of the keys, unused
    order  [Bs, H, n_cap]                int32: the slot of each position in time, a permutation
    count  [Bs, H]                       int32: chunks held
    weight [Bs, H, n_cap]                float32: accumulated gates, by position in time
"""
import math

import torch

own = False

STORED = {"int8": (torch.int8, 127.0), "e4m3": (torch.float8_e4m3fn, 448.0)}  # dtype, largest value
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
C = 64  # tokens per chunk
TINY = 2.0 ** -100  # a block whose largest magnitude is below this is stored as zeros


# ------------------------------------------------------------------------------- cases
def _decode(name, Bs, H, dk, dv, n, n_rep, fmt, dtype, ragged=False, evicted=False, active=0.0, gdn2=False):
    return dict(name=name, op="decode", Bs=Bs, H=H, dk=dk, dv=dv, n=n, n_rep=n_rep, fmt=fmt, dtype=dtype,
                ragged=ragged, evicted=evicted, active=active, gdn2=gdn2)


def _append(name, Bs, H, dk, dv, n_src, n_cap, n_rep, fmt, dtype, kind):
    return dict(name=name, op="append", Bs=Bs, H=H, dk=dk, dv=dv, n_src=n_src, n_cap=n_cap, n_rep=n_rep, fmt=fmt,
                dtype=dtype, kind=kind)


def listed():
    return [
        # one short conversation: the latency of a single decode step
        _decode("decode_short", 1, 16, 128, 128, 8, 2, "int8", "bf16"),
        # a full serving batch, 64 chunks each, scored by the chunks' own keys
        _decode("decode_batch", 256, 16, 128, 128, 64, 64, "int8", "bf16"),
        # one document of 65536 tokens: few rows, the longest chain a call accepts
        _decode("decode_long", 1, 16, 128, 128, 1024, 2, "int8", "bf16"),
        # requests of every length, the caller's gates, most chunks below the threshold, after evictions
        _decode("decode_skip", 33, 5, 64, 128, 200, 3, "e4m3", "f32", ragged=True, evicted=True, active=0.25),
        # the channel-wise recurrence, mixed lengths
        _decode("decode_gdn2", 48, 16, 128, 64, 96, 17, "e4m3", "bf16", ragged=True, evicted=True, gdn2=True),
        # a prompt of 32768 tokens enters the cache whole
        _append("fill_prompt", 1, 16, 128, 128, 512, 512, 64, "int8", "bf16", "fill"),
        # what eviction kept of four prompts enters a small cache, float32 maps
        _append("fill_selected", 4, 6, 64, 64, 128, 32, 5, "e4m3", "f32", "selected"),
        # the live chunks of a batch are complete: each full cache drops one chunk and takes the new one
        _append("commit_batch", 64, 16, 128, 128, 1, 16, 2, "int8", "f32", "commit"),
        # the weights that a prompt's own gates give its chunks: 65536 tokens, and a batch of mixed lengths
        dict(name="weights_long", op="weights", Bs=1, H=16, n=1024, ragged=False),
        dict(name="weights_batch", op="weights", Bs=21, H=16, n=125, ragged=True),
        # a prompt's chunks cut to a budget, and the step that makes room for one chunk
        dict(name="evict_prompt", op="evict", Bs=8, H=16, n=1024, budget=256, n_recent=16, ragged=False),
        dict(name="evict_step", op="evict", Bs=256, H=16, n=64, budget=63, n_recent=4, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "decode", "append", "append", "weights", "evict"])
    H = rng.choice([1, 2, 3, 4, 5, 6, 8, 11, 16])
    if op == "decode":
        n = _log_int(rng, 1, 1024)
        rows = _log_int(rng, 1, max(1, min(4096, 100_000 // n)))
        active = rng.choice([0.0, 0.0, 0.25, 0.6])
        case = _decode("", max(1, rows // H), H, rng.choice([64, 128]), rng.choice([64, 128]), n, _log_int(rng, 1, 64),
                       rng.choice(["int8", "e4m3"]), rng.choice(["bf16", "f32"]), rng.random() < 0.5,
                       rng.random() < 0.5, active, rng.random() < 0.3)
    elif op == "append":
        kind = rng.choice(["fill", "selected", "commit"])
        n_cap = _log_int(rng, 2, 512)
        rows = _log_int(rng, 1, max(1, min(1024, 8192 // n_cap)))
        n_src = {"fill": rng.randint(1, n_cap), "selected": min(1024, n_cap + rng.randint(0, n_cap)), "commit": 1}[kind]
        case = _append("", max(1, rows // H), H, rng.choice([64, 128]), rng.choice([64, 128]), n_src, n_cap,
                       _log_int(rng, 1, 64), rng.choice(["int8", "e4m3"]),
                       "f32" if kind == "commit" else rng.choice(["bf16", "f32"]), kind)
    elif op == "weights":
        n = _log_int(rng, 8, 1024)
        case = dict(op=op, Bs=max(1, _log_int(rng, 1, max(1, min(512, 16 * 1024 * 1024 // (n * n)))) // H), H=H, n=n,
                    ragged=rng.random() < 0.5)
    else:
        n = _log_int(rng, 4, 1024)
        budget = rng.randint(1, n)
        case = dict(op=op, Bs=max(1, _log_int(rng, 1, 4096) // H), H=H, n=n, budget=budget,
                    n_recent=rng.randint(0, budget), ragged=rng.random() < 0.5)
    case.pop("name", None)
    return case


def _counts(case):
    """Chunks held per (sequence, head), summed: half of the slots where lengths are mixed."""
    rows = case["Bs"] * case["H"]
    return rows * case["n"] / (2 if case["ragged"] and rows > 1 else 1)


def work(case):
    rows = case["Bs"] * case["H"]
    op = case["op"]
    if op == "weights":
        pairs = rows * case["n"] * (case["n"] - 1) / 2 / (3 if case["ragged"] else 1)
        return {"bytes": 4 * pairs + 4 * rows * case["n"], "flops": pairs}
    if op == "evict":
        return {"bytes": 16.0 * rows * case["n"], "flops": _counts(case)}
    dk, dv, n_rep = case["dk"], case["dv"], case["n_rep"]
    maps, keys = dk * (dk + dv), n_rep * dk
    if op == "append":
        kept = rows * min(case["n_src"], case["n_cap"])
        e = 2 if case["dtype"] == "bf16" else 4
        reads = (maps + keys) * e
        writes = maps + keys + 16 + 8 + (maps * 4 if case["kind"] == "commit" else 0)
        return {"bytes": float(kept * (reads + writes)), "flops": float(3 * kept * (maps + keys))}
    held = _counts(case)
    read = held * case["active"] if case["active"] else held
    e = 2 if case["dtype"] == "bf16" else 4
    token = (2 * dk + dv) * e + (4 * (2 * dk + dv) if case["gdn2"] else 8) + 4 * dv
    scored = 0.0 if case["active"] else held * keys
    nbytes = read * (maps + 8) + scored + held * (4 + 4 + 4 + 8) + rows * (8 * maps + token)
    return {"bytes": float(nbytes), "flops": float(2 * (read * maps + scored) + 8 * rows * maps)}


# ------------------------------------------------------------------------------ inputs
def _bytes(x):
    return x.view(torch.uint8)  # 8-bit floats are indexed as bytes


def _quantise(x, fmt, dims):
    """x in 8 bits with one scale over `dims`: (values as x / scale in the stored type, scale)."""
    dtype, top = STORED[fmt]
    m = x.abs().amax(dims, keepdim=True)
    some = m >= TINY
    scale = torch.where(some, m / top, 0.0)
    y = x * torch.where(some, top / m, 0.0)
    y = y.round().clamp(-top, top) if fmt == "int8" else y.clamp(-top, top)
    return y.to(dtype), scale.flatten(-len(dims))[..., 0]


def _chunk_maps(count, dk, dv, gen):
    """Maps of `count` chunks of 64 tokens: (A [count, dk, dk], B [count, dv, dk]) float32."""
    k = torch.nn.functional.normalize(torch.randn(count, C, dk, generator=gen, device="cuda"), dim=-1)
    v = torch.randn(count, C, dv, generator=gen, device="cuda")
    beta = 0.02 + 0.18 * torch.rand(count, C, 1, 1, generator=gen, device="cuda")
    alpha = 0.997 + 0.003 * torch.rand(count, C, 1, 1, generator=gen, device="cuda")
    A = torch.eye(dk, device="cuda").repeat(count, 1, 1)
    B = torch.zeros(count, dv, dk, device="cuda")
    for t in range(C):
        kt = k[:, t, None, :]
        A = alpha[:, t] * (A - beta[:, t] * (A * kt).sum(-1, keepdim=True) * kt)
        B = alpha[:, t] * (B - beta[:, t] * (B * kt).sum(-1, keepdim=True) * kt) + beta[:, t] * v[:, t, :, None] * kt
    return A, B


def _lengths(rows, n, ragged, gen):
    """n for every row or, where ragged, every length from a full row to an empty one."""
    if not ragged:
        return torch.full((rows,), n, dtype=torch.int32, device="cuda")
    spread = torch.linspace(n, 0, rows, device="cuda").round().to(torch.int32)
    return spread[torch.randperm(rows, generator=gen, device="cuda")]


def _spread_counts(case, gen):
    return _lengths(case["Bs"] * case["H"], case["n"], case["ragged"], gen).view(case["Bs"], case["H"])


def _order(Bs, H, n, shuffled, gen):
    if shuffled:
        return torch.rand(Bs, H, n, generator=gen, device="cuda").argsort(-1).to(torch.int32)
    return torch.arange(n, dtype=torch.int32, device="cuda").repeat(Bs, H, 1)


def _empty_cache(Bs, H, n_cap, dk, dv, n_rep, fmt):
    dtype = STORED[fmt][0]
    z = lambda *shape, dtype: torch.zeros(shape, dtype=torch.uint8 if dtype.itemsize == 1 else dtype, device="cuda").view(dtype)  # noqa: E731
    return dict(maps=z(Bs, H, n_cap, dk + dv, dk, dtype=dtype), reps=z(Bs, H, n_cap, n_rep, dk, dtype=dtype),
                scale=z(Bs, H, n_cap, 4, dtype=torch.float32),
                order=torch.arange(n_cap, dtype=torch.int32, device="cuda").repeat(Bs, H, 1),
                count=z(Bs, H, dtype=torch.int32), weight=z(Bs, H, n_cap, dtype=torch.float32))


def _full_cache(case, n, shuffled, gen, q=None):
    """A cache of n slots in use.  With a query q the keys of a chunk are drawn so that its
    logit lies near a level of its own between -5 and -1: a few chunks matter to a token."""
    Bs, H, dk, dv, n_rep, fmt = (case[x] for x in ("Bs", "H", "dk", "dv", "n_rep", "fmt"))
    A, B = _chunk_maps(48, dk, dv, gen)
    a8, sa = _quantise(A - torch.eye(dk, device="cuda"), fmt, (-2, -1))
    b8, sb = _quantise(B, fmt, (-2, -1))
    bank = torch.cat([_bytes(a8), _bytes(b8)], 1)
    pick = torch.randint(0, 48, (Bs * H * n,), generator=gen, device="cuda")
    cache = dict(maps=bank[pick].view(STORED[fmt][0]).view(Bs, H, n, dk + dv, dk))
    jitter = 0.9 + 0.2 * torch.rand(Bs * H * n, 2, generator=gen, device="cuda")
    scale = torch.zeros(Bs, H, n, 4, device="cuda")
    scale[..., 0] = (sa[pick] * jitter[:, 0]).view(Bs, H, n)
    scale[..., 1] = (sb[pick] * jitter[:, 1]).view(Bs, H, n)
    reps = torch.empty(Bs, H, n, n_rep, dk, dtype=torch.uint8, device="cuda")
    for b in range(Bs):
        r = 0.3 * torch.randn(H, n, n_rep, dk, generator=gen, device="cuda")
        if q is not None:
            qb = q[b].float()
            level = -5 + 4 * torch.rand(H, n, 1, 1, generator=gen, device="cuda")
            r += level * (math.sqrt(dk) * qb / qb.square().sum(-1, keepdim=True))[:, None, None, :]
        r8, scale[b, ..., 2] = _quantise(r, fmt, (-2, -1))
        reps[b] = _bytes(r8)
    cache.update(scale=scale, reps=reps.view(STORED[fmt][0]), order=_order(Bs, H, n, shuffled, gen),
                 count=torch.full((Bs, H), n, dtype=torch.int32, device="cuda"), weight=_weights(Bs, H, n, gen))
    return cache


def _weights(Bs, H, n, gen):
    """Accumulated gates: a long tail, and chunks that no token has read yet (equal weights of zero)."""
    w = -4.0 * torch.log(torch.rand(Bs, H, n, generator=gen, device="cuda").clamp_min(1e-6))
    return torch.where(torch.rand(Bs, H, n, generator=gen, device="cuda") < 0.1, 0.0, w)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *shape: torch.rand(shape, generator=gen, device="cuda")  # noqa: E731
    randn = lambda *shape: torch.randn(shape, generator=gen, device="cuda")  # noqa: E731
    Bs, H = case["Bs"], case["H"]
    s = dict(case=case)
    if case["op"] == "weights":
        n = case["n"]
        s["gates"] = torch.sigmoid(randn(Bs, H, n, n) * 3 - 4).contiguous()
        if case["ragged"]:
            s["n_chunks"] = _lengths(Bs, n, True, gen)
        return s
    if case["op"] == "evict":
        n = case["n"]
        s.update(weight=_weights(Bs, H, n, gen), count=_spread_counts(case, gen), order=_order(Bs, H, n, True, gen),
                 out=(torch.empty(Bs, H, n, dtype=torch.int32, device="cuda"),
                      torch.empty(Bs, H, n, device="cuda"), torch.empty(Bs, H, dtype=torch.int32, device="cuda")))
        return s
    dk, dv, n_rep, fmt, dtype = case["dk"], case["dv"], case["n_rep"], case["fmt"], TYPES[case["dtype"]]
    if case["op"] == "append":
        n_src, n_cap = case["n_src"], case["n_cap"]
        if case["kind"] == "commit":
            s["cache"] = _full_cache(case, n_cap, True, gen)
        else:
            s["cache"] = _empty_cache(Bs, H, n_cap, dk, dv, n_rep, fmt)
        A, B = _chunk_maps(96, dk, dv, gen)
        pick = torch.randint(0, 96, (Bs * H * n_src,), generator=gen, device="cuda")
        spread = torch.exp(randn(Bs, H, n_src, 1, 1) * 0.5)
        s["At"] = A.transpose(-1, -2).contiguous()[pick].view(Bs, H, n_src, dk, dk).to(dtype).contiguous()
        s["Bc"] = (B.transpose(-1, -2).contiguous()[pick].view(Bs, H, n_src, dk, dv) * spread).to(dtype).contiguous()
        s["reps"] = randn(Bs, n_src * n_rep, H, dk).to(dtype)
        if case["kind"] == "selected":
            keep = rand(Bs, H, n_src).argsort(-1)[..., :n_cap].sort(-1).values
            s["src"] = torch.zeros(Bs, H, n_src, dtype=torch.int32, device="cuda")
            s["src"][..., :n_cap] = keep.to(torch.int32)
            s["n_new"] = torch.randint(0, n_cap + 1, (Bs, H), generator=gen, device="cuda", dtype=torch.int32)
            s["weight_in"] = _weights(Bs, H, n_src, gen)
    else:
        n = case["n"]
        s["q"], s["k"] = (randn(Bs, H, dk).to(dtype) for _ in range(2))
        s["k"] = torch.nn.functional.normalize(s["k"].float(), dim=-1).to(dtype)
        s["v"] = randn(Bs, H, dv).to(dtype)
        s["S_cur"], s["At_cur"] = 0.1 * randn(Bs, H, dk, dv), torch.eye(dk, device="cuda") - 0.02 * rand(Bs, H, dk, dk)
        s["cache"] = _full_cache(case, n, case["evicted"], gen, s["q"])
        s["cache"]["count"] = _spread_counts(case, gen)
        if case["gdn2"]:
            s["token_gates"] = (0.8 + 0.2 * rand(Bs, H, dk), rand(Bs, H, dk), rand(Bs, H, dv))
        else:
            s["token_gates"] = (rand(Bs, H), 0.8 + 0.2 * rand(Bs, H))
        s["tau"] = 1e-3
        if case["active"]:
            s["tau"] = 0.1
            on = rand(Bs, H, n) < case["active"]
            s["gates_in"] = torch.where(on, 0.15 + 0.8 * rand(Bs, H, n), 0.08 * rand(Bs, H, n))
        s["o"], s["gates_out"] = torch.empty(Bs, H, dv, device="cuda"), torch.empty(Bs, H, n, device="cuda")
    s["lib_cache"] = None
    return s


# -------------------------------------------------------------------------- plain forms
def _rows(cache):
    Bs, H = cache["count"].shape
    return (torch.arange(Bs, device="cuda").view(Bs, 1), torch.arange(H, device="cuda").view(1, H))


def _live_update(s):
    """The token enters the live chunk (state S_cur and transition At_cur, updated in place)."""
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    M, At = s["S_cur"], s["At_cur"]
    if s["case"]["gdn2"]:
        a, b, w = s["token_gates"]
        M.mul_(a[..., None])
        At.mul_(a[..., None])
        erase, write = b * k, w * v
    else:
        beta, alpha = (x[..., None] for x in s["token_gates"])
        M.mul_(alpha[..., None])
        At.mul_(alpha[..., None])
        erase, write = beta * k, beta * v
    M.sub_(erase[..., None] * (k[..., None] * M).sum(-2, keepdim=True)).add_(k[..., None] * write[..., None, :])
    At.sub_(erase[..., None] * (k[..., None] * At).sum(-2, keepdim=True))
    return q, (M * q[..., None]).sum(-2), (At * q[..., None]).sum(-2)


def _plain_decode(s):
    c, tau = s["cache"], s["tau"]
    dk, dtype = s["case"]["dk"], c["maps"].dtype
    q, o, z = _live_update(s)
    b, h = _rows(c)
    maps, reps = _bytes(c["maps"]), _bytes(c["reps"])
    gates_in = s.get("gates_in")
    # each chunk acts on what the later ones left: the recursion over the chunks, newest first
    for j in reversed(range(s["case"]["n"])):
        slot = c["order"][:, :, j].long()
        held = j < c["count"]
        scale = c["scale"][b, h, slot]
        if gates_in is None:
            r = reps[b, h, slot].view(dtype).float()
            score = (r * q[:, :, None, :]).sum(-1) * (scale[..., 2:3] / math.sqrt(dk))
            top = score.amax(-1)
            logit = top + (score - top[..., None]).exp().mean(-1).log()
            g = 1.0 / (1.0 + (-logit).exp())
        else:
            g = gates_in[:, :, j]
        s["gates_out"][:, :, j] = torch.where(held, g, 0.0)
        g = torch.where(held & (g >= tau), g, 0.0)
        c["weight"][:, :, j] += g.clamp(0.0, 1.0)
        y = torch.matmul(maps[b, h, slot].view(dtype).float(), z[..., None])[..., 0]
        o = o + (g * scale[..., 1])[..., None] * y[..., dk:]
        z = z + (g * scale[..., 0])[..., None] * y[..., :dk]
    s["o"].copy_(o)


def _plain_evict(weight, count, order, budget, n_recent):
    n = weight.shape[-1]
    pos = torch.arange(n, device=weight.device)
    held = pos < count[..., None]
    key = torch.where(pos < count[..., None] - n_recent, weight, math.inf)
    key = torch.where(held, key, math.nan)  # sorts last
    rank = key.argsort(stable=True, dim=-1).argsort(-1)  # lowest weight first, ties by position
    leaves = rank < (count[..., None] - budget)
    kind = torch.where(held, leaves.long(), 2)
    to = kind.argsort(stable=True, dim=-1)
    left = torch.minimum(count, torch.full_like(count, budget))
    kept = torch.where(pos < left[..., None], weight.gather(-1, to), 0.0)
    return order.gather(-1, to), kept, left


def _plain_append(s):
    c, case = s["cache"], s["case"]
    n_src, n_cap, n_rep, dk, dv, fmt = (case[x] for x in ("n_src", "n_cap", "n_rep", "dk", "dv", "fmt"))
    Bs, H = c["count"].shape
    if case["kind"] == "commit":
        order, weight, count = _plain_evict(c["weight"], c["count"], c["order"], n_cap - 1, 1)
        c["order"].copy_(order)
        c["weight"].copy_(weight)
        c["count"].copy_(count)
    else:
        c["count"].zero_()
        c["weight"].zero_()
        c["order"].copy_(torch.arange(n_cap, dtype=torch.int32, device="cuda").expand(Bs, H, n_cap))
    n_pos = min(n_src, n_cap)
    i = torch.arange(n_pos, device="cuda")
    b, h = (x[..., None] for x in _rows(c))
    src = s["src"][..., :n_pos].long() if "src" in s else i.expand(Bs, H, n_pos)
    new = s["n_new"] if "n_new" in s else torch.full((Bs, H), n_pos, dtype=torch.int32, device="cuda")
    pos = c["count"][..., None] + i
    slot = c["order"].gather(-1, pos.long()).long()
    valid = i < new[..., None]
    A = s["At"][b, h, src].transpose(-1, -2).float() - torch.eye(dk, device="cuda")
    B = s["Bc"][b, h, src].transpose(-1, -2).float()
    R = s["reps"].view(Bs, n_src, n_rep, H, dk).permute(0, 3, 1, 2, 4)[b, h, src].float()
    (a8, sa), (b8, sb), (r8, sr) = (_quantise(x, fmt, (-2, -1)) for x in (A, B, R))
    maps, reps = _bytes(c["maps"]), _bytes(c["reps"])
    at = (b, h, slot)
    wide = valid[..., None, None]
    maps[at] = torch.where(wide, torch.cat([_bytes(a8), _bytes(b8)], -2), maps[at])
    reps[at] = torch.where(wide, _bytes(r8), reps[at])
    c["scale"][at] = torch.where(valid[..., None], torch.stack([sa, sb, sr, torch.zeros_like(sa)], -1), c["scale"][at])
    fresh = s["weight_in"][..., :n_pos] if "weight_in" in s else torch.zeros(Bs, H, n_pos, device="cuda")
    c["weight"].scatter_(-1, pos.long(), torch.where(valid, fresh, 0.0))
    c["count"].add_(new)
    if case["kind"] == "commit":
        s["At"].copy_(torch.eye(dk, device="cuda").expand_as(s["At"]))
        s["Bc"].zero_()


def _plain_weights(s):
    g = s["gates"]
    n = g.shape[-1]
    i = torch.arange(n, device="cuda")
    held = torch.full((g.shape[0],), n, device="cuda") if "n_chunks" not in s else s["n_chunks"]
    on = (i[:, None] > i) & (g >= 1e-3) & (i[:, None] < held[:, None, None, None])
    return torch.where(on, g.clamp(0.0, 1.0), 0.0).sum(-2)


def run(s):
    if own:
        return _own(s)
    case = s["case"]
    if case["op"] == "weights":
        return _plain_weights(s)
    if case["op"] == "evict":
        return _plain_evict(s["weight"], s["count"], s["order"], case["budget"], case["n_recent"])
    (_plain_decode if case["op"] == "decode" else _plain_append)(s)
    return _outputs(s)


def _outputs(s):
    c = s["cache"]
    if s["case"]["op"] == "append":
        return {**c, "At": s["At"], "Bc": s["Bc"]} if s["case"]["kind"] == "commit" else c
    return dict(o=s["o"], S_cur=s["S_cur"], At_cur=s["At_cur"], gates=s["gates_out"], weight=c["weight"])


# ------------------------------------------------------------------------ the framework
def _own(s):
    from gated_deltanet_hybrid_amd import hla
    case = s["case"]
    if case["op"] == "weights":
        return hla.gate_weights(s["gates"], tau=1e-3, n_chunks=s.get("n_chunks"))
    if case["op"] == "evict":
        return hla.evict_chunks(s["weight"], s["count"], case["budget"], case["n_recent"], order=s["order"],
                                out=s["out"])
    if s["lib_cache"] is None:  # the program's cache object, around the same tensors
        s["lib_cache"] = hla.Cache8(**s["cache"])
    c = s["lib_cache"]
    if case["op"] == "append":
        commit = case["kind"] == "commit"
        if commit:
            hla.cache8_evict(c, case["n_cap"] - 1, 1)
        hla.cache8_append(c, s["At"], s["Bc"], s["reps"], src=s.get("src"), n_new=s.get("n_new"),
                          weight_in=s.get("weight_in"), reset=not commit, reset_live=commit)
    else:
        step = hla.gdn2_decode8 if case["gdn2"] else hla.gdn_decode8
        step(s["q"], s["k"], s["v"], *s["token_gates"], s["S_cur"], s["At_cur"], c, gates_in=s.get("gates_in"),
             tau=s["tau"], o=s["o"], gates_out=s["gates_out"])
    return _outputs(s)


# ------------------------------------------------------------------ the definition, 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "evict":
        return None
    if op == "weights":
        g = s["gates"].double()
        n = case["n"]
        last = s["n_chunks"].tolist() if "n_chunks" in s else [n] * case["Bs"]
        out = torch.zeros(case["Bs"], case["H"], n, dtype=torch.float64, device="cuda")
        for b, m in enumerate(last):
            kept = torch.tril(g[b, :, :m, :m], -1)
            out[b, :, :m] = (kept * (s["gates"][b, :, :m, :m] >= 1e-3)).sum(1)
        return out
    return _exact_append(s) if op == "append" else _exact_decode(s)


def _exact_append(s):
    """Scales, weights and the quotients that e4m3 rounds; what is whole has no such value."""
    c, case = s["cache"], s["case"]
    Bs, H, n_cap, n_rep, dk = (case[x] for x in ("Bs", "H", "n_cap", "n_rep", "dk"))
    n = min(case["n_src"], n_cap)
    scale, weight = c["scale"].double(), c["weight"].double()
    at = torch.arange(n, device="cuda").expand(Bs, H, n)
    taken, valid = at, torch.ones(Bs, H, n, dtype=torch.bool, device="cuda")
    if case["kind"] == "selected":
        taken, valid = s["src"][..., :n].long(), at < s["n_new"][..., None]
        weight[..., :n] = s["weight_in"][..., :n].double() * valid
    elif case["kind"] == "commit":  # the first of the lightest chunks leaves; its slot takes the new one
        pos = torch.arange(n_cap, device="cuda")
        older = weight[..., :-1]
        first = torch.where(older == older.min(-1, keepdim=True).values, pos[:-1], n_cap).min(-1, keepdim=True).values
        at = c["order"].gather(-1, first).long()
        weight = weight.gather(-1, (pos + (pos >= first)).clamp(max=n_cap - 1)) * (pos < n_cap - 1)
    pick = lambda x: x.gather(2, taken[..., None, None].expand(Bs, H, n, *x.shape[3:]))  # noqa: E731
    E = pick(s["At"]).double().mT - torch.eye(dk, dtype=torch.float64, device="cuda")
    B = pick(s["Bc"]).double().mT
    R = pick(s["reps"].view(Bs, case["n_src"], n_rep, H, dk).permute(0, 3, 1, 2, 4)).double()
    unit = torch.stack([x.abs().flatten(-2).max(-1).values for x in (E, B, R)], -1) / STORED[case["fmt"]][1]
    put = lambda x, new, m: x.scatter(2, at.view(Bs, H, n, *(1,) * (x.dim() - 3)).expand_as(new),  # noqa: E731
                                      torch.where(m, new, x.gather(2, at.view(Bs, H, n, *(1,) * (x.dim() - 3)).expand_as(new))))
    scale[..., :3] = put(scale[..., :3], unit, valid[..., None])
    out = dict(maps=None, reps=None, scale=scale, order=None, count=None, weight=weight)
    if case["fmt"] == "e4m3":
        wide = valid[..., None, None]
        unit = unit[..., None, None]
        out["maps"] = put(c["maps"].double(), torch.cat([E / unit[..., 0, :, :], B / unit[..., 1, :, :]], -2), wide)
        out["reps"] = put(c["reps"].double(), R / unit[..., 2, :, :], wide)
    if case["kind"] == "commit":
        out["At"] = torch.eye(dk, dtype=torch.float64, device="cuda").expand_as(s["At"])
        out["Bc"] = torch.zeros_like(s["Bc"], dtype=torch.float64)
    return out


def _exact_decode(s):
    """The states composed oldest first, S -> S + g (S E + B), then read with y: the definition."""
    c, case = s["cache"], s["case"]
    Bs, H, dk, dv, n = (case[x] for x in ("Bs", "H", "dk", "dv", "n"))
    f8 = c["maps"].dtype
    q, k, v = (s[x].double() for x in ("q", "k", "v"))
    S, A = s["S_cur"].double().mT, s["At_cur"].double().mT  # [dv, dk], [dk, dk]
    if case["gdn2"]:
        a, er, wr = (x.double() for x in s["token_gates"])
        S, A, er, wr = S * a[:, :, None], A * a[:, :, None], er * k, wr * v
    else:
        beta, alpha = (x.double()[:, :, None] for x in s["token_gates"])
        S, A, er, wr = S * alpha[..., None], A * alpha[..., None], beta * k, beta * v
    S = S - (S @ k[..., None]) * er[:, :, None] + wr[..., None] * k[:, :, None]
    A = A - (A @ k[..., None]) * er[:, :, None]
    y = A @ q[..., None]
    held = torch.arange(n, device="cuda") < c["count"][..., None]
    slot = c["order"].long()
    scale = c["scale"].double().gather(2, slot[..., None].expand(Bs, H, n, 4))
    if "gates_in" in s:
        g = s["gates_in"].double()
    else:
        g = torch.zeros(Bs, H, n, dtype=torch.float64, device="cuda")
        for b in range(Bs):
            r = _bytes(c["reps"])[b].gather(1, slot[b][..., None, None].expand(H, n, case["n_rep"], dk))
            e = ((r.view(f8).double() @ q[b][:, None, :, None])[..., 0] * scale[b, ..., 2:3] / math.sqrt(dk)).exp()
            m = e.mean(-1)
            g[b] = m / (1 + m)
    kept = torch.where(held & (g >= s["tau"]), g, 0.0)
    past = torch.zeros(Bs, H, dv, dk, dtype=torch.float64, device="cuda")
    b, h = _rows(c)
    for j in range(n):
        m = _bytes(c["maps"])[b, h, slot[:, :, j]].view(f8).double()
        ga, gb = ((kept[:, :, j] * scale[:, :, j, i])[..., None, None] for i in (0, 1))
        past = past + ga * (past @ m[:, :, :dk]) + gb * m[:, :, dk:]
    o = (S @ q[..., None] + past @ y)[..., 0]
    return dict(o=o, S_cur=S.mT, At_cur=A.mT, gates=torch.where(held, g, 0.0),
                weight=c["weight"].double() + kept.clamp(0, 1))
