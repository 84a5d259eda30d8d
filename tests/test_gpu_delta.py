"""The gated delta rule, its gradient and its single-token form against the float64 oracle on the GPU.

Tolerances, derived before the first run, in u = 2^-24 (an fp32 rounding) and half a step of the output type.
- Inputs are those of the layer: keys and queries of length 1, beta in (0, 1), decays at most 1. A token's step
  a (I - beta k k^T) then lengthens no vector, so an error made at one token is carried on at most at its size, and errors
  of different tokens and terms are independent: they add as root sums of squares.
- A result passes at most 8 products one after the other (K S, T R, the inverse itself, K^T u; in the gradient as many
  again), each a sum of at most 128 products in order: sqrt(128 / 3) u = 6.5 u relative to the sum's terms, sqrt(8) of
  those 18.5 u. Terms exceed their sums by up to about 4 here (an error V - G K S, a difference of reads): 74 u. With exps
  and the join of pieces (8 u each) below 96 u of a head's norm.
- So fp32 results: norm of the error at most 96 u of the norm, head by head, and no value off by more than 8 times the
  head's root mean square share of that (the largest of 10^5 normal values is below 5) on top of 96 u of its own.
- bf16 results: half a step (2^-8 relative) on top, value by value; and o, dq and dk are made of operands in two bf16
  parts. The first part is off by 2^-9 of the value at most and the second by 2^-9 of that: 2^-18. A product of two such
  operands is off by 2^-18 for each and by 2^-18 for the product of their second parts, which is left out: 3 * 2^-18 of the
  product's magnitude. `_terms` sums those magnitudes for every value of o, dq and dk (with |x . y| at most |x| |y| for
  the sums over a head's channels).
"""
import numpy as np
import pytest
import torch

import test_layer_amd as tla
from gpu_util import to64
from oracle import delta

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def _close(got, want, heads_axis_shape=None, names="", terms=None):
    """got (a tensor) against want (float64), head by head: axis 1 of `heads_axis_shape`."""
    x, y = to64(got), np.asarray(want)
    parts = np.zeros_like(y) if terms is None or got.dtype == torch.float32 else 3 * 2.0 ** -18 * terms
    shape = heads_axis_shape or (len(y), 1, -1)
    x, y, parts = x.reshape(shape), y.reshape(shape), parts.reshape(shape)
    half = HALF[got.dtype]
    for h in range(y.shape[1]):
        a, b = x[:, h], y[:, h]
        live = ~np.isnan(b)
        a, b, more = a[live], b[live], parts[:, h][live]
        if not b.size:
            continue
        rms = np.sqrt(np.mean(b * b))
        err = np.abs(a - b)
        assert np.isfinite(a).all(), (names, h)
        far = err - (96 * U + half) * np.abs(b) - 8 * 96 * U * rms - more
        assert (far <= 0).all(), (names, h, float(err.max()), float(rms))
        if got.dtype == torch.float32 and b.size >= 64:
            assert np.linalg.norm(a - b) <= 96 * U * np.linalg.norm(b), (names, h, np.linalg.norm(a - b) / np.linalg.norm(b) / U)


def _case(lens, hk, group, dk, dv, dtype, gate=True, state=True, seed=0, behind=0):
    g = np.random.default_rng(seed)
    n, hv, dt = sum(lens), hk * group, DT[dtype]

    def unit(d):
        x = g.standard_normal((n, hk, d))
        return x / np.maximum(np.linalg.norm(x, axis=-1, keepdims=True), 1e-12)

    def t(x, dt=torch.float32):
        x = torch.tensor(x, dtype=torch.float32).flatten(1).to(dt)
        if behind:  # rows of no sequence
            x = torch.cat([x, torch.full((behind, x.shape[1]), float("nan"), dtype=dt)])
        return x.cuda()

    c = dict(q=t(unit(dk), dt), k=t(unit(dk), dt), v=t(g.standard_normal((n, hv * dv)), dt), heads=hk,
             g=t(-np.exp(g.standard_normal((n, hv)) * 1.5 - 2)) if gate else None, beta=t(g.uniform(0.02, 0.98, (n, hv))),
             cu=torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda(), lens=lens, dims=(hv, dk, dv),
             do=t(g.standard_normal((n, hv * dv)), dt), n=n)
    shape = (len(lens), hv, dk, dv)
    c["state"] = torch.tensor(g.standard_normal(shape) * 0.3, dtype=torch.float32).cuda() if state else None
    c["dstate"] = torch.tensor(g.standard_normal(shape) * 0.3, dtype=torch.float32).cuda() if state else None
    return c


def _np(t, n):
    return None if t is None else to64(t)[:n]


def _oracle(c, scale=1.0, grad=False):
    n = c["n"]
    a = [_np(c[x], n) for x in ("q", "k", "v", "g", "beta")]
    S = None if c["state"] is None else to64(c["state"])
    cu = c["cu"].cpu().numpy()
    if not grad:
        return delta.run(*a, c["heads"], S, scale, cu)
    return delta.run(*a, c["heads"], S, scale, cu, _np(c["do"], n), None if c["dstate"] is None else to64(c["dstate"]))


def _terms(c, scale, grad):
    """Magnitudes of the terms of o (or of dq and dk), chunk by chunk of 32 tokens, laid out as they are."""
    n, (hv, dk, dv), hk = c["n"], c["dims"], c["heads"]
    q, k, v, do = (_np(c[x], n).reshape(n, -1, d) for x, d in (("q", dk), ("k", dk), ("v", dv), ("do", dv)))
    beta = _np(c["beta"], n)
    a = np.exp(_np(c["g"], n)) if c["g"] is not None else np.ones_like(beta)
    o, dq, dkk = np.zeros((n, hv, dv)), np.zeros((n, hk, dk)), np.zeros((n, hk, dk))
    norm = lambda x, axis=-1: np.sqrt((x * x).sum(axis))  # noqa: E731
    for b, h in np.ndindex(len(c["lens"]), hv):
        lo, hi = int(c["cu"][b]), int(c["cu"][b + 1])
        kh = h // (hv // hk)
        Q, K, V, DO, B, A = q[lo:hi, kh], k[lo:hi, kh], v[lo:hi, h], do[lo:hi, h], beta[lo:hi, h], a[lo:hi, h]
        S = np.zeros((dk, dv)) if c["state"] is None else to64(c["state"])[b, h]
        Ss, us = [], []
        for t in range(hi - lo):
            Ss.append(S)
            S = A[t] * S
            us.append(B[t] * (V[t] - S.T @ K[t]))
            S = S + np.outer(K[t], us[-1])
        if not grad:
            for t in range(hi - lo):
                first = t - t % 32
                o[lo + t, h] = scale * norm(Q[t]) * (norm(Ss[first], 0) + sum(np.abs(us[j]) * norm(K[j]) for j in range(first, t + 1)))
            continue
        dS = np.zeros((dk, dv)) if c["dstate"] is None else to64(c["dstate"])[b, h]
        dSs, dR = [None] * (hi - lo), [None] * (hi - lo)
        for t in reversed(range(hi - lo)):
            dSs[t] = dS  # after token t
            dS = dS + scale * np.outer(Q[t], DO[t])
            dR[t] = B[t] * (dS.T @ K[t])
            dS = A[t] * (dS - np.outer(K[t], dR[t]))
        for t in range(hi - lo):
            first, last = t - t % 32, min(hi - lo, t - t % 32 + 32) - 1
            S0, S1 = norm(Ss[first]), norm(dSs[last])
            dq[lo + t, kh] += scale * norm(DO[t]) * (S0 + sum(norm(us[j]) * np.abs(K[j]) for j in range(first, t + 1)))
            dkk[lo + t, kh] += norm(us[t]) * S1 + norm(dR[t]) * S0
            dkk[lo + t, kh] += sum(scale * norm(DO[i]) * norm(us[t]) * np.abs(Q[i]) for i in range(t, last + 1))
            dkk[lo + t, kh] += sum(norm(dR[t]) * norm(us[j]) * np.abs(K[j]) for j in range(first, t))
            dkk[lo + t, kh] += sum(norm(dR[i]) * norm(us[t]) * np.abs(K[i]) for i in range(t + 1, last + 1))
    return {"dq": dq.reshape(n, -1), "dk": dkk.reshape(n, -1)} if grad else o.reshape(n, -1)


def _forward(c, scale=1.0, **kw):
    return tla.gated_delta(c["q"], c["k"], c["v"], c["g"], c["beta"], c["heads"], scale, c["state"], c["cu"], **kw)


def _grad(c, scale=1.0, **kw):
    return tla.gated_delta_grad(c["q"], c["k"], c["v"], c["g"], c["beta"], c["do"], c["heads"], c["dstate"], scale, c["state"],
                                c["cu"], **kw)


def _check_forward(c, scale=1.0, **kw):
    o, S = _forward(c, scale, **kw)
    hv, dk, dv = c["dims"]
    n = c["n"]
    want_o, want_S = _oracle(c, scale)
    if n:
        _close(o[:n], want_o, (n, hv, dv), "o", _terms(c, scale, False) if o.dtype == torch.bfloat16 else None)
    _close(S, want_S, (len(c["lens"]), hv, dk * dv), "state")
    return o, S


def _check_grad(c, scale=1.0, **kw):
    got = _grad(c, scale, **kw)
    want = _oracle(c, scale, True)
    terms = _terms(c, scale, True) if c["q"].dtype == torch.bfloat16 else {}
    hv, dk, dv = c["dims"]
    n, hk = c["n"], c["heads"]
    shapes = dict(dq=(n, hk, dk), dk=(n, hk, dk), dv=(n, hv, dv), dg=(n, hv, 1), dbeta=(n, hv, 1), dstate=(len(c["lens"]), hv, dk * dv))
    for name, t in got._asdict().items():
        if t is None:
            assert name == "dg" and c["g"] is None or name == "dstate" and c["state"] is None
        elif t.numel():
            _close(t if name == "dstate" else t[:n], want[name], shapes[name], name, terms.get(name))
    return got


DIMS = [(64, 64), (128, 64), (64, 128), (128, 128)]
LENS = [[1], [31, 32, 33], [0, 5, 0], [64, 1, 0, 95, 96, 97], [200], [3] * 70]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_forward(lens, dk, dv, dtype):
    _check_forward(_case(lens, 2, 1 if dk == dv else 2, dk, dv, dtype, seed=sum(lens)), 1.0 if dk == 64 else 0.3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate,state", [(False, True), (True, False), (False, False)])
def test_forward_without_gate_or_state(gate, state, dtype):
    _check_forward(_case([70, 40], 3, 1, 64, 64, dtype, gate, state, 5))


# Sequences long enough to be cut into pieces (of 3 chunks = 96 tokens at these sizes, where longer than 240), with piece ends
# inside a chunk.
LONG = [[129], [128], [700], [300, 0, 1, 513, 40], [1374]]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("lens", LONG, ids=str)
def test_forward_in_pieces(lens, dk, dv, dtype):
    if sum(lens) > 1000 and dk != dv:
        lens = [900, 17]
    c = _case(lens, 1, 2, dk, dv, dtype, state=len(lens) != 1 or lens[0] != 700, seed=sum(lens))
    o, S = _check_forward(c)
    # told that no sequence is long, the same sequences are not cut: another order of the same sums
    o1, S1 = _check_forward(c, max_seqlen=1)
    _close(S, to64(S1), (len(lens), 2, dk * dv), "uncut")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_grad(lens, dk, dv, dtype):
    _check_grad(_case(lens, 2, 1 if dk == dv else 2, dk, dv, dtype, seed=sum(lens)), 1.0 if dk == 64 else 0.3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("lens", LONG, ids=str)
def test_grad_in_pieces(lens, dk, dv, dtype):
    if sum(lens) > 1000 and dk != dv:
        lens = [900, 17]
    _check_grad(_case(lens, 1, 1, dk, dv, dtype, seed=sum(lens)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate,state", [(False, True), (True, False), (False, False)])
def test_grad_without_gate_or_state(gate, state, dtype):
    _check_grad(_case([150, 40], 2, 3, 64, 64, dtype, gate, state, 6), 0.5)


def _copies(c, times):
    """The case with its heads `times` over."""
    def t(x, heads):
        return None if x is None else x.reshape(len(x), heads, -1).repeat(1, times, 1).flatten(1)

    hk, (hv, dk, dv) = c["heads"], c["dims"]
    m = dict(c, heads=hk * times, dims=(hv * times, dk, dv))
    for name, heads in (("q", hk), ("k", hk), ("v", hv), ("do", hv), ("g", hv), ("beta", hv)):
        m[name] = t(c[name], heads)
    for name in ("state", "dstate"):
        m[name] = None if c[name] is None else c[name].repeat(1, times, 1, 1)
    return m


# Enough chunks x heads for waves of 64 columns (32 where d_k is 128), with sequences that are cut and that are not.
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("lens", [[1450, 5, 0, 700], [1050, 1051]], ids=str)
def test_many_heads_in_wide_waves(lens, dk, dv, dtype, monkeypatch):
    one = _case(lens, 1, 2 if dk != dv else 1, dk, dv, dtype, seed=dk + dv)
    times = 256 * 64 // dv // one["dims"][0]
    many = _copies(one, times)
    n, (hv, _, _), hk = one["n"], one["dims"], 1

    def first(x, heads):  # every copy's bits are the first one's
        if x.dim() == 4:
            y = x.reshape(len(x), times, heads, dk, dv)
        else:
            y = x.reshape(n, times, heads, -1)
        assert torch.equal(y, y[:, :1].expand_as(y))
        return y[:, 0].contiguous() if x.dim() == 4 else y[:, 0].flatten(1)

    o, S = _forward(many)
    got = _grad(many)
    heads = dict(dq=hk, dk=hk, dv=hv, dg=hv, dbeta=hv, dstate=hv)
    monkeypatch.setattr(tla, "gated_delta", lambda *a, **k: (first(o, hv), first(S, hv)))
    monkeypatch.setattr(tla, "gated_delta_grad",
                        lambda *a, **k: tla.GatedDeltaGrads(*[first(t, heads[name]) for name, t in got._asdict().items()]))
    _check_forward(one)
    _check_grad(one)


def test_many_heads_and_a_whole_view():
    _check_forward(_case([1374], 16, 1, 64, 64, "bf16", seed=1))
    _check_grad(_case([400, 333], 16, 1, 64, 64, "bf16", seed=2))


def test_shared_heads_over_many_rows():
    # a shared key head's gradients are the sums, in their order, of those of as many key heads of the same rows
    c = _case([40000, 0, 26001], 1, 2, 64, 64, "f32", seed=7, behind=5)
    got = _grad(c)
    apart = _grad(dict(c, q=c["q"].repeat(1, 2), k=c["k"].repeat(1, 2), heads=2))
    n = c["n"]
    for name in ("dq", "dk"):
        a = getattr(apart, name)[:n]
        assert torch.equal(getattr(got, name)[:n], a[:, :64] + a[:, 64:]), name
    assert torch.equal(got.dv[:n], apart.dv[:n]) and torch.equal(got.dbeta[:n], apart.dbeta[:n])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_thousands_of_sequences(dtype):
    lens = np.random.default_rng(8).integers(0, 3, 5000).tolist()
    lens[4100] = 70
    c = _case(lens, 1, 1, 64, 64, dtype, state=False, seed=8)
    _check_forward(c)
    _check_grad(c)


def test_a_head_is_its_own():
    c = _case([200, 77], 3, 2, 64, 64, "bf16", seed=3)
    o, S = _forward(c)
    for h in range(6):
        kh = h // 2
        one = dict(c, q=c["q"][:, kh * 64:kh * 64 + 64].contiguous(), k=c["k"][:, kh * 64:kh * 64 + 64].contiguous(),
                   v=c["v"][:, h * 64:h * 64 + 64].contiguous(), g=c["g"][:, h:h + 1].contiguous(),
                   beta=c["beta"][:, h:h + 1].contiguous(), state=c["state"][:, h:h + 1].contiguous(), heads=1)
        o1, S1 = _forward(one, max_seqlen=1)
        o2, S2 = _forward(c, max_seqlen=1)
        assert torch.equal(o1, o2[:, h * 64:h * 64 + 64]) and torch.equal(S1[:, 0], S2[:, h])


def test_decays_of_every_size():
    # no decay, total decay (-Inf), and ones far past fp32's exponents, next to ordinary ones
    c = _case([150, 90], 1, 4, 64, 64, "f32", seed=4)
    g = c["g"]
    g[::7] = 0.0
    g[20] = g[64] = g[95] = g[180] = -float("inf")
    g[33:36, 1] = -1e30
    g[70:90, 2] = -50.0
    g[100, 3] = -1e4
    _check_forward(c)
    got = _check_grad(c)
    assert torch.isfinite(got.dg).all()
    # what lies before a total decay does not count at all
    for x in ("q", "k", "v"):
        c[x][:20] *= 3
    o, S = _forward(c)
    c["state"][0] = 7.0
    o2, S2 = _forward(c)
    assert torch.equal(o[96:150], o2[96:150]) and torch.equal(S, S2)


def test_repeated_keys():
    # the same key over and over at a full step: the triangle of ones, whose inverse repeated squaring would lose
    c = _case([200], 1, 1, 64, 64, "f32", gate=False, seed=5)
    c["k"][:] = c["k"][:1].clone()
    c["beta"][:] = 1.0
    o, S = _forward(c)
    k = c["k"][:1]
    assert torch.allclose(S[0, 0].T @ k[0], c["v"][-1], atol=1e-5)
    _check_forward(c)
    _check_grad(c)


@pytest.mark.parametrize("beta", [0.0, 1.0])
def test_no_step_and_full_steps(beta):
    c = _case([90, 40], 2, 1, 64, 64, "f32", seed=6)
    c["beta"][:] = beta
    _check_forward(c)
    got = _check_grad(c)
    if beta == 0.0:
        assert (got.dv == 0).all() and not (got.dbeta == 0).all()


def test_zero_keys_and_queries():
    c = _case([90], 2, 1, 64, 64, "bf16", seed=7)
    for x in ("q", "k"):
        c[x][10:50] = 0
    o, _ = _check_forward(c)
    assert (o[10:50] == 0).all()
    got = _check_grad(c)
    assert torch.isfinite(got.dk).all()


def test_rows_of_no_sequence_are_neither_read_nor_written():
    for behind in (1, 31, 40):
        c = _case([50, 45], 1, 2, 64, 64, "bf16", seed=behind, behind=behind)
        keep = torch.full_like(c["v"], 5.0)
        o, S = _check_forward(c, out=keep)
        assert o is keep and (o[c["n"]:] == 5.0).all() and torch.isfinite(S).all()
        out = tla.GatedDeltaGrads(*(torch.full_like(c[x], 5.0) for x in ("q", "k", "v", "g", "beta")), torch.empty_like(S))
        got = _check_grad(c, out=out)
        for x in got[:5]:
            assert (x[c["n"]:] == 5.0).all()


def test_gaps_between_sequences_as_sequences():
    # a sequence whose rows hold NaN spoils itself alone
    c = _case([40, 20, 70], 2, 1, 64, 64, "f32", seed=8)
    o, S = _forward(c, max_seqlen=1)
    got = _grad(c, max_seqlen=1)
    for x in ("q", "k", "v", "g", "beta", "do"):
        c[x][40:60] = float("nan")
    o2, S2 = _forward(c, max_seqlen=1)
    got2 = _grad(c, max_seqlen=1)
    for a, b in zip((o, *got[:5]), (o2, *got2[:5])):
        assert torch.equal(a[:40], b[:40]) and torch.equal(a[60:], b[60:])
    assert torch.equal(S[[0, 2]], S2[[0, 2]]) and torch.isnan(S2[1]).any()


def test_boundaries_outside_the_rows():
    c = _case([40, 37], 1, 1, 64, 64, "bf16", seed=9)
    o, S = _forward(c)
    for cu in ([-5, 40, 1000], [0, 40, 2 ** 31 - 1]):
        bad = dict(c, cu=torch.tensor(cu, dtype=torch.int32).cuda())
        o2, S2 = _forward(bad)
        assert torch.equal(o, o2) and torch.equal(S, S2)
        assert torch.equal(_grad(bad).dk, _grad(c).dk)
    back = dict(c, cu=torch.tensor([0, 40, 40], dtype=torch.int32).cuda())
    back2 = dict(c, cu=torch.tensor([0, 40, 10], dtype=torch.int32).cuda())  # ends before it begins: empty
    keep, keep2 = torch.zeros_like(o), torch.zeros_like(o)
    _, S1 = _forward(back, out=keep)
    _, S2 = _forward(back2, out=keep2)
    assert torch.equal(keep, keep2) and torch.equal(S1, S2) and torch.equal(S1[1], c["state"][1])


def test_no_tokens():
    c = _case([0, 0], 2, 2, 64, 64, "bf16", seed=1)
    o, S = _forward(c)
    assert o.shape == (0, 256) and torch.equal(S, c["state"])
    got = _grad(c)
    assert torch.equal(got.dstate, c["dstate"]) and got.dq.shape == (0, 128)
    c["state"] = c["dstate"] = None
    assert (_forward(c)[1] == 0).all()
    out = tla.gated_delta_step(c["q"], c["k"], c["v"], c["g"], c["beta"], 2, torch.zeros(3, 4, 64, 64, device="cuda"))
    assert out.shape == (0, 256)


def test_one_sequence_without_boundaries():
    c = _case([333], 2, 1, 64, 64, "bf16", seed=2)
    o, S = _forward(c)
    o2, S2 = tla.gated_delta(c["q"], c["k"], c["v"], c["g"], c["beta"], 2, state=c["state"])
    assert torch.equal(o, o2) and torch.equal(S, S2)
    a, b = _grad(c), _grad(dict(c, cu=None))
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_state_in_place_and_given_outputs_and_same_bits():
    for lens in ([100, 30], [700, 30]):
        c = _case(lens, 1, 2, 64, 128, "bf16", seed=3)
        o, S = _forward(c)
        got = _grad(c)
        ws = torch.empty(tla.gated_delta_workspace_bytes(sum(lens), 2, 0, 1, 2, 64, 128, tla.BF16) + 64, dtype=torch.uint8,
                         device="cuda")
        ws[:] = 0xFF  # NaN: nothing of it is read before it is written
        st = c["state"].clone()
        out = torch.empty_like(o)
        o2, S2 = tla.gated_delta(c["q"], c["k"], c["v"], c["g"], c["beta"], 1, state=st, cu_seqlens=c["cu"], out=out, state_out=st,
                                 workspace=ws)
        assert o2 is out and S2 is st and torch.equal(o, o2) and torch.equal(S, S2)
        need = tla.gated_delta_grad_workspace_bytes(sum(lens), 2, 0, 1, 2, 64, 128, tla.BF16)
        ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")
        ds = c["dstate"].clone()
        again = _grad(dict(c, dstate=ds), out=got._replace(**{k: torch.empty_like(v) for k, v in got._asdict().items()},
                                                           )._replace(dstate=ds), workspace=ws)
        assert again.dstate is ds and all(torch.equal(x, y) for x, y in zip(got, again))
        assert (ws[need:] == 0xFF).all()


def test_unwanted_gradients_are_left_alone():
    c = _case([90, 50], 1, 2, 64, 64, "bf16", seed=4)
    got = _grad(c)
    for name in tla.GatedDeltaGrads._fields:
        one = tla.GatedDeltaGrads(**{name: torch.empty_like(getattr(got, name))})
        _grad(c, out=one)
        assert torch.equal(getattr(one, name), getattr(got, name)), name
    c = _case([90, 50], 2, 1, 64, 64, "f32", seed=5)
    got = _grad(c)
    for name in ("dq", "dk", "dstate"):
        one = tla.GatedDeltaGrads(**{name: torch.empty_like(getattr(got, name))})
        _grad(c, out=one)
        assert torch.equal(getattr(one, name), getattr(got, name)), name


def test_gradient_against_differences_of_the_forward():
    # fp32 forward at step 2^-7 along a random direction: central differences are off by the third derivative, h^2 / 6 of
    # the loss's scale (below 2^-16 of it here), and by its rounding, 96 u / h = 2^-10 of it
    c = _case([75], 1, 1, 64, 64, "f32", seed=6)
    gen = torch.Generator("cuda").manual_seed(0)
    do, dS = torch.randn(c["v"].shape, generator=gen, device="cuda"), torch.randn(c["state"].shape, generator=gen, device="cuda")
    c["do"], c["dstate"] = do, dS
    got = _grad(c)

    def loss(x):
        o, S = _forward(x)
        return float((o.double() * do.double()).sum() + (S.double() * dS.double()).sum())

    for name, grad in (("q", got.dq), ("k", got.dk), ("v", got.dv), ("g", got.dg), ("beta", got.dbeta), ("state", got.dstate)):
        way = torch.randn(c[name].shape, generator=gen, device="cuda")
        way /= way.norm()
        h = 2.0 ** -7
        num = (loss(dict(c, **{name: c[name] + h * way})) - loss(dict(c, **{name: c[name] - h * way}))) / (2 * h)
        want = float((grad.double() * way.double()).sum())
        assert abs(num - want) <= 2.0 ** -9 * (abs(want) + float(grad.double().norm())), name


# ----------------------------------------------------------------------------------------------------- single tokens

def _step(c, rows, state, slots=None, scale=1.0):
    a = [None if c[x] is None else c[x][rows].contiguous() for x in ("q", "k", "v", "g", "beta")]
    return tla.gated_delta_step(*a, c["heads"], state, slots, scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("rows,gate", [(1, True), (5, False), (67, True), (300, True)])
def test_step(rows, gate, dk, dv, dtype):
    group = 1 if dk == dv else 2
    c = _case([1] * rows, 2, group, dk, dv, dtype, gate, True, rows)
    want_o, want_S = _oracle(c, 0.7)
    state = c["state"].clone()
    o = _step(c, slice(None), state, scale=0.7)
    _close(o, want_o, (rows, 2 * group, dv), "o")
    _close(state, want_S, (rows, 2 * group, dk * dv), "state")
    # the same states in another order of a larger cache
    perm = torch.randperm(rows + 9, generator=torch.Generator().manual_seed(0))[:rows].to(torch.int32).cuda()
    cache = torch.full((rows + 9, 2 * group, dk, dv), 3.0, device="cuda")
    cache[perm.long()] = c["state"]
    o2 = _step(c, slice(None), cache, perm, 0.7)
    assert torch.equal(o, o2) and torch.equal(cache[perm.long()], state)
    rest = torch.ones(rows + 9, dtype=torch.bool, device="cuda")
    rest[perm.long()] = False
    assert (cache[rest] == 3.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_steps_one_by_one_are_the_sequence(dtype):
    c = _case([70], 2, 2, 64, 64, dtype, seed=1)
    want_o, want_S = _oracle(c)
    state = c["state"].clone()
    o = torch.cat([_step(c, slice(t, t + 1), state) for t in range(70)])
    _close(o, want_o, (70, 4, 64), "o")
    _close(state, want_S, (1, 4, 64 * 64), "state")
    # all 70 as rows of one slot
    state2 = c["state"].clone()
    o2 = _step(c, slice(None), state2, torch.zeros(70, dtype=torch.int32, device="cuda"))
    assert torch.equal(o, o2) and torch.equal(state, state2)


def test_rows_of_one_slot_in_their_order():
    # 600 rows on 7 slots, more rows than a workgroup looks at at once; some left out
    c = _case([600], 1, 1, 64, 64, "f32", seed=2)
    gen = torch.Generator().manual_seed(1)
    slots = torch.randint(0, 7, (600,), generator=gen).to(torch.int32)
    slots[::11] = -1
    slots[5] = 7
    slots[599] = 2 ** 31 - 1
    slots[6] = -2 ** 31
    first = torch.randn(7, 1, 64, 64, generator=gen).cuda() * 0.3
    state = first.clone()
    o = _step(c, slice(None), state, slots.cuda())
    out = (slots < 0) | (slots >= 7)
    assert (o[out.cuda()] == 0).all()
    for s in range(7):
        rows = (slots == s).nonzero()[:, 0].cuda()
        want = first[s:s + 1].clone()
        w = torch.cat([_step(c, rows[i:i + 1], want) for i in range(len(rows))])
        assert torch.equal(o[rows], w) and torch.equal(state[s:s + 1], want)


def test_no_slot_at_all():
    c = _case([4], 1, 1, 64, 64, "bf16", seed=3)
    state = torch.zeros(0, 1, 64, 64, device="cuda")
    o = _step(c, slice(None), state, torch.zeros(4, dtype=torch.int32, device="cuda"))
    assert (o == 0).all()


def test_prefill_then_steps():
    # a view's tokens at once, then the next tokens one by one: the sequence's own results
    c = _case([150], 2, 1, 64, 64, "bf16", seed=4)
    want_o, want_S = _oracle(c)
    cut = {x: (None if c[x] is None else c[x][:100].contiguous()) for x in ("q", "k", "v", "g", "beta")}
    o, state = tla.gated_delta(*cut.values(), 2, state=c["state"])
    steps = [_step(c, slice(t, t + 1), state) for t in range(100, 150)]
    _close(torch.cat([o, *steps]), want_o, (150, 2, 64), "o")
    _close(state, want_S, (1, 2, 64 * 64), "state")


# --------------------------------------------------------------------------------- streams, graphs, far addresses

def test_another_stream_and_two_at_once():
    cs = [_case([500, 33], 1, 2, 64, 64, d, seed=i) for i, d in enumerate(("bf16", "f32"))]
    want = [(_forward(c), _grad(c)) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for c, s in zip(cs, streams):
        with torch.cuda.stream(s):
            got.append((_forward(c), _grad(c)))
    torch.cuda.synchronize()
    for (f, b), (f2, b2) in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip((*f, *b), (*f2, *b2)))


def test_captured_and_replayed():
    c = _case([500, 33], 1, 2, 64, 64, "bf16", seed=1)
    s = _case([1] * 5, 1, 2, 64, 64, "bf16", seed=2)
    state = torch.zeros(5, 2, 64, 64, device="cuda")
    for x in range(2):  # warm, on the stream that captures
        _forward(c), _grad(c), _step(s, slice(None), state)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for i in range(2):  # two graphs over the same inputs, each with memory of its own
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f, b = _forward(c), _grad(c)
            o = _step(s, slice(None), state)
        graphs.append(g)
        outs.append((*f, *b, o))
    own = torch.zeros_like(state)
    state.zero_()
    for turn in range(4):
        c["v"].copy_(torch.randn_like(c["v"]))
        c["do"].copy_(torch.randn_like(c["do"]))
        graphs[turn % 2].replay()
        graphs[1 - turn % 2].replay()
        torch.cuda.synchronize()
        want = (*_forward(c), *_grad(c))
        _step(s, slice(None), own)
        mid = _step(s, slice(None), own)
        for got in outs:
            assert all(torch.equal(x, y) for x, y in zip(got, want)), turn
        assert torch.equal(state, own) and torch.equal(outs[1 - turn % 2][-1], mid)


def test_more_than_2_31_values_and_a_far_slot():
    # 2.2 million tokens of 16 heads: offsets past 2^31 values and 2^32 bytes, in sequences of about a view's length
    n, C = 2_200_000, 1024
    cu = torch.arange(0, n, 1374, dtype=torch.int32)
    cu = torch.cat([cu, torch.tensor([n], dtype=torch.int32)]).cuda()
    gen = torch.Generator("cuda").manual_seed(0)
    q, k = (torch.nn.functional.normalize(torch.randn(n, 16, 64, generator=gen, device="cuda", dtype=torch.bfloat16), dim=-1)
            .flatten(1) for _ in range(2))
    v = torch.randn(n, C, generator=gen, device="cuda", dtype=torch.bfloat16)
    g = -torch.rand(n, 16, generator=gen, device="cuda") * 0.1
    beta = torch.rand(n, 16, generator=gen, device="cuda")
    o, S = tla.gated_delta(q, k, v, g, beta, 16, cu_seqlens=cu, max_seqlen=1374)
    lo = int(cu[-3])
    part = [t[lo:].contiguous() for t in (q, k, v, g, beta)]
    o2, S2 = tla.gated_delta(*part, 16, cu_seqlens=cu[-3:] - lo, max_seqlen=1)  # uncut, as among that many sequences
    assert n * C > 2 ** 31
    assert torch.equal(o[lo:], o2) and torch.equal(S[-2:], S2)
    del o, q, k, v, g, beta
    state = torch.zeros(33000, 16, 64, 64, device="cuda")
    assert state.numel() > 2 ** 31
    first = torch.randn(1, 16, 64, 64, device="cuda")
    state[32999] = first
    row = [t[:1].contiguous() for t in part]
    o3 = tla.gated_delta_step(*row, 16, state, torch.tensor([32999], dtype=torch.int32, device="cuda"))
    o4 = tla.gated_delta_step(*row, 16, first)
    assert torch.equal(o3, o4) and torch.equal(state[32999:], first) and (state[:32999].amax() == 0)
