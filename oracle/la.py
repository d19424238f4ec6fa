"""Linear attention with a decay for each head, token by token in float64: one head's
M_t = exp(g_t) M_{t-1} + k_t v_t^T, o_t = M_t^T q_t and the gradients by the reverse recurrence
G_t = exp(g_{t+1}) G_{t+1} + q_t do_t^T.  Layouts: M [dk, dv], tokens [T, width], g [T]."""
import numpy as np


def la_recurrent(q, k, v, g, S0=None):
    """(o [T, dv], M [T + 1, dk, dv]: the state in front of the first token and behind every one)."""
    T, dk, dv = len(g), k.shape[-1], v.shape[-1]
    M = np.zeros((T + 1, dk, dv))
    if S0 is not None:
        M[0] = S0
    o = np.zeros((T, dv))
    for t in range(T):
        M[t + 1] = np.exp(g[t]) * M[t] + np.outer(k[t], v[t])
        o[t] = q[t] @ M[t + 1]
    return o, M


def la_backward(q, k, v, g, dO, dS=None, S0=None):
    """dict(dq, dk, dv, dg, dS0) of sum(o dO) + sum(M_T dS)."""
    T = len(g)
    _, M = la_recurrent(q, k, v, g, S0)
    G = np.zeros(M.shape[1:]) if dS is None else np.array(dS, np.float64)
    out = dict(dq=np.zeros_like(q), dk=np.zeros_like(k), dv=np.zeros_like(v), dg=np.zeros(T))
    for t in reversed(range(T)):
        G = G + np.outer(q[t], dO[t])
        out["dq"][t] = M[t + 1] @ dO[t]
        out["dk"][t] = G @ v[t]
        out["dv"][t] = G.T @ k[t]
        G = np.exp(g[t]) * G
        out["dg"][t] = np.sum(G * M[t])
    out["dS0"] = G
    return out
