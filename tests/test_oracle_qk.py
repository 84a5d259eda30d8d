"""Pins of the query/key oracle: complex products, torch's norms, distances alone, and gradients against differences."""
import numpy as np
import pytest
import torch

from oracle import qk


def test_interleaved_rotation_is_a_complex_product():
    g = np.random.default_rng(0)
    x, pos = g.standard_normal((5, 2, 8)), g.integers(-50, 50, (5, 1))
    y = qk.rotate(x, pos, (4,), 100.0, True, True)
    f = 100.0 ** -(np.arange(4) / 4)
    z = (x[..., 0::2] + 1j * x[..., 1::2]) * np.exp(1j * pos * f)[:, None]
    assert np.allclose(y[..., 0::2], z.real) and np.allclose(y[..., 1::2], z.imag)


def test_halves_are_interleaved_pairs_in_another_order():
    g = np.random.default_rng(1)
    x, pos = g.standard_normal((5, 1, 8)), g.integers(-50, 50, (5, 1))
    order = np.array([0, 4, 1, 5, 2, 6, 3, 7])
    a = qk.rotate(x, pos, (4,), 100.0, True, False)
    b = qk.rotate(x[..., order], pos, (4,), 100.0, True, True)
    assert np.allclose(a[..., order], b)


@pytest.mark.parametrize("per_axis", [True, False])
@pytest.mark.parametrize("interleaved", [True, False])
def test_products_see_distances_alone(per_axis, interleaved):
    g = np.random.default_rng(2)
    q, k = g.standard_normal((2, 1, 1, 14))
    sec = (2, 3, 1)
    rot = lambda x, p: qk.rotate(x, np.array([p]), sec, 30.0, per_axis, interleaved)  # noqa: E731
    d = [np.sum(rot(q, p) * rot(k, np.add(p, (3, -1, 4)))) for p in ((0, 0, 0), (5, 9, -2), (1000, 1, 7))]
    assert np.allclose(d, d[0], rtol=1e-10)
    assert np.allclose(rot(q, (4, 5, 6))[..., 12:], q[..., 12:])  # channels behind the sections
    assert np.allclose(np.linalg.norm(rot(q, (4, 5, 6))), np.linalg.norm(q))


def test_norms_match_torch():
    x = np.random.default_rng(3).standard_normal((5, 24)) + 0.7
    w, b = np.random.default_rng(4).standard_normal((2, 24))
    t = torch.tensor
    assert np.allclose(qk.norm(x, "l2", eps=1e-12)[0], torch.nn.functional.normalize(t(x), dim=-1).numpy())
    assert np.allclose(qk.norm(x, "rms", w)[0], torch.nn.functional.rms_norm(t(x), (24,), t(w), 1e-6).numpy())
    assert np.allclose(qk.norm(x, "layer", w, b)[0], torch.nn.functional.layer_norm(t(x), (24,), t(w), t(b), 1e-6).numpy())
    assert np.allclose(qk.norm(np.full((1, 4), 1e-3), "l2", eps=1.0)[0], 1e-3)


@pytest.mark.parametrize("kind", ["none", "l2", "l2short", "rms", "layer"])
def test_gradients_against_differences(kind):
    g = np.random.default_rng(5)
    n, heads, d = 3, 2, 6
    x, dy = g.standard_normal((2, n, heads * d))
    w, b = (g.standard_normal((2, d)) if kind in ("rms", "layer") else (None, None))
    pos = g.integers(0, 9, (n, 2))
    eps = 50.0 if kind == "l2short" else 1e-6
    rest = dict(eps=eps, pos=pos, sections=(1, 2), base=20.0, per_axis=True, interleaved=False)
    kind = kind[:2] if kind == "l2short" else kind
    dx, dw, db = qk.grads(x, dy, heads, kind, w, **rest)
    for name, v, got in (("x", x, dx), ("w", w, dw), ("b", b, db)):
        if v is None:
            continue
        num = np.zeros_like(v)
        for i in np.ndindex(v.shape):
            lim = []
            for s in (1e-6, -1e-6):
                p = dict(x=x, w=w, b=b)
                p[name] = v.copy()
                p[name][i] += s
                lim.append((qk.forward(p["x"], heads, kind, p["w"], p["b"], **rest) * dy).sum())
            num[i] = (lim[0] - lim[1]) / 2e-6
        assert np.allclose(got, num, rtol=1e-6, atol=1e-7), name
