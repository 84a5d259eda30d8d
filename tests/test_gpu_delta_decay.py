"""The gradient of the gated delta rule's decays where these are strong, head by head, against the float64 oracle on the GPU.

dg_t = <dP_t, P_t> with P_t = e^{g_t} S_{t-1} the decayed state and dP_t its gradient: however small e^{g_t}, both are results
of the rule, right to 96 u of their norms (u = 2^-24; the derivation stands in test_gpu_delta.py), so every value of dg is
right to 2 * 96 u |dP_t| |P_t|, and in one head, where all decays are alike, dg to 96 u of its norm as other results are.
"""
import numpy as np
import pytest
import torch

import test_layer_amd as tla

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _case(lens, dk, dv, dtype, gates, seed):
    """A head for each of gates(n) -> [n]."""
    r = np.random.default_rng(seed)
    n, heads = sum(lens), len(gates)

    def t(x):
        return torch.tensor(x, dtype=torch.float32).flatten(1).to(DT[dtype]).cuda()

    def unit(d):
        x = r.standard_normal((n, heads, d))
        return t(x / np.linalg.norm(x, axis=-1, keepdims=True))

    g = torch.tensor(np.stack([f(n) for f in gates], 1), dtype=torch.float32).cuda()
    state, dstate = (torch.tensor(r.standard_normal((len(lens), heads, dk, dv)) * 0.3, dtype=torch.float32).cuda() for _ in range(2))
    return dict(q=unit(dk), k=unit(dk), v=t(r.standard_normal((n, heads, dv))), g=g, do=t(r.standard_normal((n, heads, dv))),
                beta=torch.tensor(r.uniform(0.02, 0.98, (n, heads)), dtype=torch.float32).cuda(), state=state, dstate=dstate,
                cu=torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda())


def _want(c, dk, dv):
    """(dg, |dP| |P|), token by token in 64 bits."""
    q, k, v, g, beta, do, S0, S1 = (c[x].double().cpu().numpy() for x in ("q", "k", "v", "g", "beta", "do", "state", "dstate"))
    n, heads = g.shape
    q, k, v, do = (x.reshape(n, heads, -1) for x in (q, k, v, do))
    dg, size = np.empty((n, heads)), np.empty((n, heads))
    cu = c["cu"].tolist()
    for b, h in np.ndindex(len(cu) - 1, heads):
        S, kept = S0[b, h], []
        for t in range(cu[b], cu[b + 1]):
            P = np.exp(g[t, h]) * S
            kept.append(P)
            S = P + np.outer(k[t, h], beta[t, h] * (v[t, h] - P.T @ k[t, h]))
        dS = S1[b, h]
        for t in reversed(range(cu[b], cu[b + 1])):
            dS = dS + np.outer(q[t, h], do[t, h])
            dP = dS - np.outer(k[t, h], beta[t, h] * (dS.T @ k[t, h]))
            P = kept[t - cu[b]]
            dg[t, h], size[t, h] = np.sum(dP * P), np.linalg.norm(dP) * np.linalg.norm(P)
            dS = np.exp(g[t, h]) * dP
    return dg, size


def _grad(c):
    heads = c["g"].shape[1]
    return tla.gated_delta_grad(c["q"], c["k"], c["v"], c["g"], c["beta"], c["do"], heads, dstate=c["dstate"], state=c["state"],
                                cu_seqlens=c["cu"])


def _check(c, dk, dv):
    got = _grad(c).dg.double().cpu().numpy()
    want, size = _want(c, dk, dv)
    err = np.abs(got - want)
    assert (err <= 192 * U * size).all(), float((err - 192 * U * size).max())
    return got, want


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 64), (64, 128), (128, 128)])
@pytest.mark.parametrize("lens", [[75], [31, 33, 1], [300, 40]], ids=str)
def test_heads_of_one_decay(lens, dk, dv, dtype):
    sizes = (-1e-3, -3.0, -8.0, -12.0, -20.0, -50.0)
    c = _case(lens, dk, dv, dtype, [lambda n, x=x: np.full(n, x) for x in sizes], sum(lens))
    got, want = _check(c, dk, dv)
    for h, g in enumerate(sizes):
        err = np.linalg.norm(got[:, h] - want[:, h]) / np.linalg.norm(want[:, h])
        assert err <= 96 * U, (g, err / U)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
def test_strong_decays_among_weak_ones(dk, dv, dtype):
    def every(m, strong, weak=-0.01):
        return lambda n: np.where(np.arange(n) % m == m - 1, strong, weak)

    c = _case([120, 50], dk, dv, dtype, [every(2, -20.0), every(7, -30.0), every(32, -12.0), every(5, -1e4), every(3, -float("inf"))], 3)
    got, _ = _check(c, dk, dv)
    assert (got[2::3, 4][:39] == 0).all()  # a token that forgets everything: 0, not what is left of a difference


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [0.3, 3.0, 20.0, 80.0])
@pytest.mark.parametrize("n", [2, 32, 45])
def test_decays_between_two_tokens(n, size, dtype):
    # key 0 at a full step, read n - 1 tokens later, and the state: the decays of all tokens between, spread over 512 heads.
    # A decay is two exps of 2 u and their product; up to 45 logarithms add in two floats (the lower ones below 2^-7 a token:
    # 1 u in all), and a chunk's end is one more product: 8 u of the value at every size
    heads = 512
    g = torch.zeros(n, heads)
    g[1:] = -torch.rand(n - 1, heads, generator=torch.Generator().manual_seed(n)) * size / (n - 1)
    q, k = torch.zeros(n, heads, 64), torch.zeros(n, heads, 64)
    q[-1, :, 0] = 1.0
    k[torch.arange(n), :, torch.arange(n)] = 1.0
    rows = [x.flatten(1).to(DT[dtype]).cuda() for x in (q, k, torch.ones(n, heads, 64))]
    o, state = tla.gated_delta(*rows, g.cuda(), torch.ones(n, heads, device="cuda"), heads)
    want = torch.exp(g.double().sum(0))
    # bf16: a value below 2^-110 has parts below 2^-126, the least normal number, which count as 0: 2^-126 for each of two
    half, least = (2.0 ** -8, 2.0 ** -125) if dtype == "bf16" else (0.0, 0.0)
    assert ((state[0, :, 0, 0].double().cpu() - want).abs() <= 8 * U * want + least).all()
    assert ((o.view(n, heads, 64)[-1, :, 0].double().cpu() - want).abs() <= (8 * U + half) * want + least).all()
