"""Plain numpy oracle of the gated delta rule and its gradient (float64, no shared code with the HIP path).

    S <- e^g S,  u = beta (v - S^T k),  S <- S + k u^T,  o = scale S^T q

token by token, for one value head of one sequence: q, k [n, d_k], v [n, d_v], g, beta [n], S [d_k, d_v].
"""
from __future__ import annotations

import numpy as np


def forward(q, k, v, g, beta, S=None, scale=1.0):
    """(o [n, d_v], the last state)."""
    n, dk, dv = len(q), q.shape[1], v.shape[1]
    S = np.zeros((dk, dv)) if S is None else np.array(S, np.float64)
    o = np.empty((n, dv))
    for t in range(n):
        S = np.exp(g[t]) * S
        S = S + np.outer(k[t], beta[t] * (v[t] - S.T @ k[t]))
        o[t] = scale * (S.T @ q[t])
    return o, S


def grads(q, k, v, g, beta, do, S=None, dS=None, scale=1.0):
    """Gradients of sum(o do) + sum(last state dS), as a dict."""
    n, dk, dv = len(q), q.shape[1], v.shape[1]
    S = np.zeros((dk, dv)) if S is None else np.array(S, np.float64)
    kept = []
    for t in range(n):
        P = np.exp(g[t]) * S
        u = beta[t] * (v[t] - P.T @ k[t])
        S = P + np.outer(k[t], u)
        kept.append((P, u, S))
    dS = np.zeros((dk, dv)) if dS is None else np.array(dS, np.float64)
    out = {"dq": np.empty((n, dk)), "dk": np.empty((n, dk)), "dv": np.empty((n, dv)), "dg": np.empty(n), "dbeta": np.empty(n)}
    for t in reversed(range(n)):
        P, u, S = kept[t]
        out["dq"][t] = scale * (S @ do[t])
        dS = dS + scale * np.outer(q[t], do[t])
        du = dS.T @ k[t]
        out["dbeta"][t] = du @ (v[t] - P.T @ k[t])
        out["dv"][t] = beta[t] * du
        out["dk"][t] = dS @ u - P @ out["dv"][t]
        dP = dS - np.outer(k[t], out["dv"][t])
        out["dg"][t] = np.sum(dP * P)
        dS = np.exp(g[t]) * dP
    out["dstate"] = dS
    return out


def _spread(x, heads, d):
    return np.asarray(x, np.float64).reshape(len(x), heads, d)


def run(q, k, v, g, beta, heads, S=None, scale=1.0, cu=None, do=None, dS=None):
    """forward (without do) or grads over sequences and heads, in the layout of the rows [n, heads * d]:
    (o, states) or a dict; rows of no sequence are NaN."""
    n, hv = beta.shape
    dk, dv, group = q.shape[1] // heads, v.shape[1] // hv, hv // heads
    cu = [0, n] if cu is None else list(cu)
    q, k, v = _spread(q, heads, dk), _spread(k, heads, dk), _spread(v, hv, dv)
    g = np.zeros((n, hv)) if g is None else np.asarray(g, np.float64)
    o = np.full((n, hv, dv), np.nan)
    last = np.empty((len(cu) - 1, hv, dk, dv))
    out = {"dq": np.full((n, heads, dk), np.nan), "dk": np.full((n, heads, dk), np.nan), "dv": np.full((n, hv, dv), np.nan),
           "dg": np.full((n, hv), np.nan), "dbeta": np.full((n, hv), np.nan), "dstate": np.empty_like(last)}
    for b, (lo, hi) in enumerate(zip(cu, cu[1:])):
        for name in ("dq", "dk"):
            out[name][lo:hi] = 0
        for h in range(hv):
            kh, s = h // group, slice(lo, hi)
            a = (q[s, kh], k[s, kh], v[s, h], g[s, h], beta[s, h].astype(np.float64))
            S0 = None if S is None else S[b, h]
            if do is None:
                o[s, h], last[b, h] = forward(*a, S0, scale)
                continue
            d = grads(*a, _spread(do, hv, dv)[s, h], S0, None if dS is None else dS[b, h], scale)
            out["dq"][s, kh] += d["dq"]
            out["dk"][s, kh] += d["dk"]
            out["dv"][s, h], out["dg"][s, h], out["dbeta"][s, h], out["dstate"][b, h] = d["dv"], d["dg"], d["dbeta"], d["dstate"]
    if do is None:
        return o.reshape(n, -1), last
    return {name: x if name in ("dg", "dbeta", "dstate") else x.reshape(n, -1) for name, x in out.items()}
