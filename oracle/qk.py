"""Plain numpy oracle of the query/key preparation (float64, no shared code with the HIP path): a norm of each head,
then the rotation of its channels by the token's position on several axes; and the gradient.
"""
from __future__ import annotations

import numpy as np


def pairs(sections, per_axis, interleaved):
    """(first channel, second channel, axis, exponent) of every rotated pair; its frequency is base^-exponent."""
    out, total = [], sum(sections)
    for a, c in enumerate(sections):
        before = sum(sections[:a])
        for j in range(c):
            i, size, off = (j, c, 2 * before) if per_axis else (before + j, total, 0)
            ch = (off + 2 * i, off + 2 * i + 1) if interleaved else (off + i, off + i + size)
            out.append((*ch, a, i / size))
    return out


def rotate(x, pos, sections, base, per_axis, interleaved, back=False):
    """x [n, heads, d] rotated (back: by the negative angles)."""
    y = np.array(x, np.float64)
    for a, b, axis, e in pairs(sections, per_axis, interleaved):
        t = (pos[:, axis].astype(np.float64) * base ** -e)[:, None] * (-1.0 if back else 1.0)
        y[..., a], y[..., b] = x[..., a] * np.cos(t) - x[..., b] * np.sin(t), x[..., b] * np.cos(t) + x[..., a] * np.sin(t)
    return y


def norm(x, kind, w=None, b=None, eps=1e-6):
    """(result, x-hat, factor) over the last axis."""
    x = np.asarray(x, np.float64)
    if kind == "none":
        return x, x, np.ones(x.shape[:-1] + (1,))
    if kind == "layer":
        x = x - x.mean(-1, keepdims=True)
    with np.errstate(all="ignore"):
        if kind == "l2":
            r = 1.0 / np.maximum(np.sqrt((x * x).sum(-1, keepdims=True)), eps)
        else:
            r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        hat = x * r
    y = hat if w is None else hat * w
    return (y if b is None else y + b), hat, r


def forward(x, heads, kind, w=None, b=None, eps=1e-6, pos=None, sections=(), base=100.0, per_axis=True, interleaved=False):
    """x [n, heads * d] -> the same."""
    n = len(x)
    y = norm(np.asarray(x, np.float64).reshape(n, heads, -1), kind, w, b, eps)[0]
    if sections:
        y = rotate(y, pos, sections, base, per_axis, interleaved)
    return y.reshape(n, -1)


def grads(x, dy, heads, kind, w=None, eps=1e-6, pos=None, sections=(), base=100.0, per_axis=True, interleaved=False):
    """(dx, dw, db)."""
    n = len(x)
    x3, d = (np.asarray(t, np.float64).reshape(n, heads, -1) for t in (x, dy))
    if sections:
        d = rotate(d, pos, sections, base, per_axis, interleaved, back=True)
    _, hat, r = norm(x3, kind, eps=eps)
    dw, db = (d * hat).sum((0, 1)), d.sum((0, 1))
    if kind == "none":
        return d.reshape(n, -1), dw, db
    d = d * (1.0 if w is None else w)
    if kind == "l2":
        free = np.sqrt((x3 * x3).sum(-1, keepdims=True)) > eps
        g = d - np.where(free, hat * (d * hat).sum(-1, keepdims=True), 0.0)
    else:
        g = d - hat * (d * hat).mean(-1, keepdims=True)
        if kind == "layer":
            g = g - d.mean(-1, keepdims=True)
    return (g * r).reshape(n, -1), dw, db
