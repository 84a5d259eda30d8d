"""Pins of the block-join oracle: torch's own norms, and every gradient against central differences."""
import numpy as np
import pytest
import torch

from oracle import join


def test_norms_match_torch():
    v = np.random.default_rng(0).standard_normal((5, 24)) + 0.7
    w, b = np.random.default_rng(1).standard_normal((2, 24))
    t = torch.tensor
    ln = torch.nn.functional.layer_norm(t(v), (24,), t(w), t(b), 1e-6).numpy()
    rms = torch.nn.functional.rms_norm(t(v), (24,), t(w), 1e-6).numpy()
    assert np.allclose(join.norm(v, "layer", w, b)[0], ln, rtol=1e-12, atol=1e-12)
    assert np.allclose(join.norm(v, "rms", w)[0], rms, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("pre", ["none", "rms", "layer"])
@pytest.mark.parametrize("per", [0, 1, 3])
def test_gradients_against_differences(post, pre, per):
    g = np.random.default_rng(7)
    n, C = 5, 6
    p = {k: g.standard_normal((n, C)) for k in ("x", "f")}
    p["scale"] = g.standard_normal(C)
    if per:
        p["gate"] = g.standard_normal((-(-n // per), C))
    if post != "none":
        p["post_w"], p["post_b"] = g.standard_normal((2, C))
    if pre != "none":
        p["pre_w"], p["pre_b"] = g.standard_normal((2, C))
    dr, dy = g.standard_normal((2, n, C))

    def loss(q):
        r = join.join(q["x"], q["f"], q.get("gate"), per or 1, q["scale"], post, q.get("post_w"), q.get("post_b"))
        L = (r * dr).sum()
        if pre != "none":
            L += (join.norm(r, pre, q["pre_w"], q["pre_b"])[0] * dy).sum()
        return L

    r = join.join(p["x"], p["f"], p.get("gate"), per or 1, p["scale"], post, p.get("post_w"), p.get("post_b"))
    got = join.grads(r, p["f"], dr, dy if pre != "none" else None, p.get("gate"), per or 1, p["scale"], post,
                     p.get("post_w"), p.get("post_b"), pre, p.get("pre_w"))
    for name, v in p.items():
        num = np.zeros_like(v)
        for i in np.ndindex(v.shape):
            q = dict(p, **{name: v.copy()})
            q[name][i] += 1e-6
            hi = loss(q)
            q[name][i] -= 2e-6
            num[i] = (hi - loss(q)) / 2e-6
        # central differences at 1e-6: truncation ~1e-12, rounding ~1e-16 / 1e-6 of a loss of order 10
        assert np.allclose(got["d" + name], num, rtol=1e-6, atol=1e-7), name
