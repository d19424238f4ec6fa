"""Inputs, float64 values and bounds for the tests of linear attention with a decay for each head.

Bounds.  Every output is a sum of products; A, the same recurrence over the inputs' magnitudes, is the
sum of the magnitudes.  A float32 sum of n terms is off by at most 6 standard deviations of n
roundings of half a step (2^-24 of a partial sum, which is below A): 6 sqrt(n / 3) 2^-24 A.  A decay
exp(x) is rounded from x in float32 and by the exponential: for the x that matter (e^-16 = 2^-24 and up)
16 + 2 steps of 2^-24, 24 with the products by it.  Over bf16 tensors the decayed scores and
the states that outputs read are rounded to 2^-16 of a term, and the output to 2^-8 of itself."""
import numpy as np
import torch

from oracle import la as ola

U = 2.0 ** -24


def steps(n):
    return (6.0 * np.sqrt(n / 3.0) + 24.0) * U


def bound(dtype, ref, mag, n):
    b = steps(n) * mag + 1e-37
    return b + 2.0 ** -8 * np.abs(ref) + 2.0 ** -15 * mag if dtype == "bf16" else b


class Case:
    """Random tokens of a padded batch, on the GPU and in float64."""

    def __init__(self, B, T, H, Hk, dk, dv, dtype, per_head=False, lens=None, start=True, ld_T=None, decay="slow", seed=0):
        r = np.random.default_rng([seed, B, T, H, dk, dv])
        ld = ld_T or T
        self.B, self.T, self.H, self.Hk, self.dk, self.dv, self.dtype = B, T, H, Hk, dk, dv, dtype
        td = torch.bfloat16 if dtype == "bf16" else torch.float32

        def tokens(*shape):
            return torch.from_numpy(r.standard_normal(shape).astype(np.float32)).to(td)

        unit = lambda x: torch.nn.functional.normalize(x.float(), dim=-1).to(td)  # noqa: E731
        self.q_, self.k_ = unit(tokens(B, ld, Hk, dk)), unit(tokens(B, ld, Hk, dk))
        self.v_, self.dO_ = tokens(B, ld, H, dv), tokens(B, T, H, dv)
        x = r.standard_normal((H,) if per_head else (B, ld, H))
        shift = {"slow": -3.0, "fast": 2.0, "none": -30.0}[decay]
        g = -np.logaddexp(0.0, x + shift)
        if not per_head and decay != "none":
            g[r.random(g.shape) < 0.02] = -np.inf
        self.g_ = torch.from_numpy(g.astype(np.float32))
        self.lens = lens
        f = lambda: torch.from_numpy(r.standard_normal((B, H, dk, dv)).astype(np.float32))  # noqa: E731
        self.S0_, self.dS_ = (f(), f()) if start else (None, None)

    def device(self, name):
        t = getattr(self, name + "_")
        if t is None:
            return None
        t = t.cuda()
        return t[:, :self.T] if name in ("q", "k", "v") or (name == "g" and t.dim() == 3) else t

    def args(self):
        return tuple(self.device(n) for n in ("q", "k", "v", "g"))

    def kw(self):
        lens = None if self.lens is None else torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        return dict(S0=self.device("S0"), lens=lens)

    def rows(self):
        """(b, h, tokens, dict of one head's arrays in float64)."""
        num = lambda t: t.float().numpy().astype(np.float64)  # noqa: E731
        q, k, v, g, dO = (num(getattr(self, n + "_")) for n in ("q", "k", "v", "g", "dO"))
        g = np.maximum(g, -1e4)
        group = self.H // self.Hk
        for b in range(self.B):
            n = self.T if self.lens is None else min(max(self.lens[b], 0), self.T)
            for h in range(self.H):
                gg = np.full(n, g[h]) if g.ndim == 1 else g[b, :n, h]
                yield b, h, n, dict(q=q[b, :n, h // group], k=k[b, :n, h // group], v=v[b, :n, h], g=gg, dO=dO[b, :n, h],
                                    S0=None if self.S0_ is None else num(self.S0_)[b, h],
                                    dS=None if self.dS_ is None else num(self.dS_)[b, h])

    def forward(self):
        """(o, S_final) in float64 and the sums of magnitudes."""
        o = np.zeros((2, self.B, self.T, self.H, self.dv))
        S = np.zeros((2, self.B, self.H, self.dk, self.dv))
        for b, h, n, x in self.rows():
            for i, f in enumerate((lambda y: y, np.abs)):
                oo, M = ola.la_recurrent(f(x["q"]), f(x["k"]), f(x["v"]), x["g"], None if x["S0"] is None else f(x["S0"]))
                o[i, b, :n, h], S[i, b, h] = oo, M[-1]
        return o, S

    def backward(self):
        """Gradients in float64 and the sums of magnitudes, as dicts of [2, ...] arrays."""
        B, T, H, Hk, dk, dv = self.B, self.T, self.H, self.Hk, self.dk, self.dv
        out = dict(dq=np.zeros((2, B, T, Hk, dk)), dk=np.zeros((2, B, T, Hk, dk)), dv=np.zeros((2, B, T, H, dv)),
                   dlog_decay=np.zeros((2, B, T, H)), dS0=np.zeros((2, B, H, dk, dv)))
        group = H // Hk
        for b, h, n, x in self.rows():
            for i, f in enumerate((lambda y: None if y is None else y, lambda y: None if y is None else np.abs(y))):
                args = [f(x[m]) for m in ("q", "k", "v")] + [x["g"], f(x["dO"]), f(x["dS"]), f(x["S0"])]
                d = ola.la_backward(*args)
                out["dq"][i, b, :n, h // group] += d["dq"]
                out["dk"][i, b, :n, h // group] += d["dk"]
                out["dv"][i, b, :n, h] = d["dv"]
                # the call sums differences of whole sums, so the largest <G, M> of the row counts
                whole = np.max(d["dg"] / np.maximum(np.exp(x["g"]), 1e-30), initial=0.0) if i else None
                out["dlog_decay"][i, b, :n, h] = whole if i else d["dg"]
                out["dS0"][i, b, h] = d["dS0"]
        if self.g_.dim() == 1:
            s = out["dlog_decay"].sum(2).sum(1)
            out["dlog_decay"] = s
        return out


def check(got, ref, mag, dtype, n, what):
    got = got.float().cpu().numpy().astype(np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    err, lim = np.abs(got - ref), bound(dtype, ref, mag, n)
    bad = ~(err <= lim)
    worst = np.max(err / lim, initial=0.0)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} beyond the bound, worst {worst:.2f} at {np.argwhere(bad)[0]}"
    return worst
