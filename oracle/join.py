"""Plain numpy oracle of the block join and its gradient (float64, no shared code with the HIP path).

    h = post(f),  r = x + scale * gate * h,  y = pre(r)

with post, pre "none", "rms" or "layer"; row t // per of gate serves token t.
"""
from __future__ import annotations

import numpy as np


def norm(v, kind, w=None, b=None, eps=1e-6):
    """(normed v, v-hat, 1/deviation) row by row."""
    v = np.asarray(v, np.float64)
    if kind == "none":
        return v, v, np.ones((v.shape[0], 1))
    if kind == "layer":
        v = v - v.mean(1, keepdims=True)
    with np.errstate(all="ignore"):
        rstd = 1.0 / np.sqrt((v * v).mean(1, keepdims=True) + eps)
        hat = v * rstd
    y = hat if w is None else hat * w
    return (y if b is None else y + b), hat, rstd


def spread(gate, per, n):
    return 1.0 if gate is None else np.repeat(np.asarray(gate, np.float64), min(per, n), axis=0)[:n]


def join(x, f, gate=None, per=1, scale=None, post="none", post_w=None, post_b=None, eps=1e-6):
    """r before it is rounded."""
    h = norm(f, post, post_w, post_b, eps)[0]
    return x + (1.0 if scale is None else scale) * spread(gate, per, len(x)) * h


def norm_back(d, hat, rstd, kind):
    """Gradient of a norm's input from that of v-hat."""
    if kind == "none":
        return d
    g = d - hat * (d * hat).mean(1, keepdims=True)
    if kind == "layer":
        g = g - d.mean(1, keepdims=True)
    return g * rstd


def grads(r, f, dr, dy, gate=None, per=1, scale=None, post="none", post_w=None, post_b=None, pre="none", pre_w=None,
          eps=1e-6):
    """All gradients, as a dict (those of absent inputs too, where they make sense)."""
    n, C = r.shape
    out = {}
    d = np.zeros((n, C)) if dr is None else np.asarray(dr, np.float64)
    if pre != "none":
        _, hat, rstd = norm(r, pre, eps=eps)
        out["dpre_w"], out["dpre_b"] = (dy * hat).sum(0), dy.sum(0)
        d = d + norm_back(dy * (1.0 if pre_w is None else pre_w), hat, rstd, pre)
    out["dx"] = d
    if f is None:
        return out
    h, hat, rstd = norm(f, post, post_w, post_b, eps)
    g, s = spread(gate, per, n), 1.0 if scale is None else scale
    out["dscale"] = (d * g * h).sum(0)
    per = min(per, n)
    groups = -(-n // per)
    p = np.zeros((groups * per, C))
    p[:n] = d * s * h
    out["dgate"] = p.reshape(groups, per, C).sum(1)
    dh = d * g * s
    out["dpost_w"], out["dpost_b"] = (dh * hat).sum(0), dh.sum(0)
    out["df"] = norm_back(dh * (1.0 if post_w is None or post == "none" else post_w), hat, rstd, post)
    return out
