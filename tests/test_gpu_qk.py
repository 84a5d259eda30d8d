"""The query/key preparation and its gradient against the float64 oracle on the GPU.

Tolerances, derived before the first run, in u = 2^-24 (an fp32 rounding) and half a step of the output type
(2^-8 relative for bf16, u for fp32):
- A head's sum adds 8 values a lane and at most 6 butterfly steps: 14 roundings, a layer norm takes two such sums; with
  the factor's square root, reciprocal and products a normed value is off by 40 u of its magnitude (|x| + mean|x|) r |w| + |b|.
- An angle is reduced to a part of a turn in 64 bits and rounded once to fp32 (2^-25 of half a turn: 2 pi 2^-26 = 1.6 u),
  sine and cosine add 2 roundings: a rotated value is off by 4 u of |a| + |b| and its three operations, 8 u in all, on top
  of the 40 u of both channels.
- A gradient goes through the rotation and two sums: 80 u of the formula with every term's magnitude in place of the term.
- Sums over tokens and heads: a lane adds its rows (at most 4 tokens x heads here), 3 butterfly steps, 4 waves, the
  workgroups' parts in 16 runs: below 128 roundings at these sizes, 128 u of the sum of magnitudes.
"""
import numpy as np
import pytest
import torch

import test_layer_amd as tla
from gpu_util import to64
from oracle import qk

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def _case(n, h, hk, d, dtype, norm, sections, per_axis, interleaved, seed=0, far=40):
    g = np.random.default_rng(seed)

    def t(*shape, std=1.0, mean=0.0, dt=torch.float32):
        return torch.tensor(g.standard_normal(shape) * std + mean, dtype=torch.float32).to(dt).cuda()

    dt = DT[dtype]
    c = dict(h=h, hk=hk, d=d, dtype=dtype, q=t(n, h * d, std=1.5, mean=0.3, dt=dt), k=t(n, hk * d, std=0.5, dt=dt) if hk else None,
             dq=t(n, h * d, dt=dt), dk=t(n, hk * d, dt=dt) if hk else None)
    for x in ("q", "k"):
        on = norm in ("rms", "layer") and (x == "q" or hk)
        c[x + "_w"] = t(d, std=0.3, mean=1.0) if on else None
        c[x + "_b"] = t(d, std=0.3) if on and norm == "layer" else None
    pos = torch.tensor(g.integers(-far, far, (n, len(sections))), dtype=torch.int32).cuda() if sections else None
    c["rest"] = dict(norm=norm, eps=1e-12 if norm == "l2" else 1e-6, pos=pos, sections=sections, base=50.0, per_axis=per_axis,
                     interleaved=interleaved)
    return c


def _forward(c, **kw):
    return tla.qk_norm_rope(c["q"], c["k"], c["h"], c["hk"] or None, q_w=c["q_w"], q_b=c["q_b"], k_w=c["k_w"], k_b=c["k_b"],
                            **c["rest"], **kw)


def _grad(c, **kw):
    return tla.qk_norm_rope_grad(c["q"], c["k"], c["dq"], c["dk"], c["h"], c["hk"] or None, q_w=c["q_w"], k_w=c["k_w"],
                                 bias=c["q_b"] is not None, **c["rest"], **kw)


def _orest(c):
    r = dict(c["rest"])
    r["kind"] = r.pop("norm")
    if r["pos"] is not None:
        r["pos"] = r["pos"].cpu().numpy()
    return r


def _f(t):
    return None if t is None else to64(t)


def _spread(m, r):
    """Magnitudes after the rotation: |a| + |b| for both channels of a pair."""
    m = np.array(m)
    for a, b, *_ in qk.pairs(r["sections"], r["per_axis"], r["interleaved"]):
        m[..., a] = m[..., b] = m[..., a] + m[..., b]
    return m


def _norm_mag(x, r, w, b):
    _, _, fac = qk.norm(x, r["kind"], eps=r["eps"])
    if r["kind"] == "none":
        return np.abs(x)
    m = (np.abs(x) + (np.abs(x).mean(-1, keepdims=True) if r["kind"] == "layer" else 0)) * fac
    m = m if w is None else m * np.abs(w)
    return m if b is None else m + np.abs(b)


def _check(c, q=None, k=None):
    got_q, got_k = _forward(c) if q is None else (q, k)
    r = _orest(c)
    for got, x, heads, w, b in ((got_q, c["q"], c["h"], c["q_w"], c["q_b"]), (got_k, c["k"], c["hk"], c["k_w"], c["k_b"])):
        if x is None:
            assert got is None
            continue
        want = qk.forward(to64(x), heads, w=_f(w), b=_f(b), **r)
        mag = _spread(_norm_mag(to64(x).reshape(len(x), heads, -1), r, _f(w), _f(b)), r).reshape(want.shape)
        tol = 48 * U * mag + HALF[c["dtype"]] * np.abs(want)
        assert (np.abs(to64(got) - want) <= tol).all()
    return got_q, got_k


def _check_grad(c, got=None):
    got = _grad(c) if got is None else got
    r = _orest(c)
    for side, x, dy, heads, w in (("q", c["q"], c["dq"], c["h"], c["q_w"]), ("k", c["k"], c["dk"], c["hk"], c["k_w"])):
        if x is None:
            assert got.dk is None and got.dk_w is None and got.dk_b is None
            continue
        x64, d64, w64 = to64(x), to64(dy), _f(w)
        dx, dw, db = qk.grads(x64, d64, heads, w=w64, **r)
        n = len(x64)
        m = _spread(np.abs(d64.reshape(n, heads, -1)), r)
        x3 = x64.reshape(n, heads, -1)
        hat = _norm_mag(x3, r, None, None)
        mw, mb = (m * hat).sum((0, 1)), m.sum((0, 1))
        if r["kind"] == "none":
            mag = m
        else:
            m = m * (1.0 if w64 is None else np.abs(w64))
            red = np.sum if r["kind"] == "l2" else np.mean
            mag = m + hat * red(m * hat, axis=-1, keepdims=True) + m.mean(-1, keepdims=True)
            mag = mag * qk.norm(x3, r["kind"], eps=r["eps"])[2]
        tol = 80 * U * mag.reshape(dx.shape) + HALF[c["dtype"]] * np.abs(dx)
        assert (np.abs(to64(getattr(got, "d" + side)) - dx) <= tol).all(), side
        for name, want, mag in (("w", dw, mw), ("b", db, mb)):
            t = getattr(got, f"d{side}_{name}")
            if t is not None:
                assert (np.abs(to64(t) - want) <= (128 + 80) * U * mag).all(), (side, name)
    return got


# norm, sections, per_axis, interleaved
KINDS = [("l2", (16, 16), True, False), ("rms", (10, 10, 10), True, False), ("layer", (8, 8), False, False),
         ("none", (16, 12, 4), False, True), ("l2", (5, 3), True, True), ("layer", (), True, False), ("rms", (7,), False, False),
         ("l2", (2, 4, 6, 20), True, False), ("none", (32,), False, False)]
SHAPES = [(1, 1, 1, 64), (5, 16, 16, 64), (70, 3, 1, 128), (33, 12, 3, 72), (9, 2, 2, 256), (3, 5, 0, 512), (40, 8, 2, 66),
          (17, 1, 4, 96), (6, 7, 7, 100), (300, 4, 4, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", KINDS, ids=str)
@pytest.mark.parametrize("n,h,hk,d", SHAPES)
def test_forward_and_gradient(n, h, hk, d, kind, dtype):
    c = _case(n, h, hk, d, dtype, *kind, seed=n + d)
    _check(c)
    _check_grad(c)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("norm", ["l2", "rms", "layer"])
@pytest.mark.parametrize("d", [1, 2, 3, 7, 31, 33, 63, 65, 127, 129, 511])
def test_odd_heads(d, norm, dtype):
    sec = (1,) if d < 4 else (d // 4, d // 8 or 1)
    sec = sec if 2 * sum(sec) <= d else ()
    c = _case(21, 3, 2, d, dtype, norm, sec, True, d % 3 == 0, seed=d)
    _check(c)
    _check_grad(c)


def test_slices_of_a_projection():
    # q and k as columns of one wider tensor, at offsets that are and are not multiples of 16 bytes (other accesses, and
    # another order of a head's sums)
    for off in (0, 8, 2, 1):
        c = _case(50, 4, 2, 64, "bf16", "rms", (16, 16), True, False, seed=off)
        wide = torch.randn(50, 1000, device="cuda").bfloat16()
        q, k = wide[:, off:off + 256], wide[:, 300 + off:300 + off + 128]
        q.copy_(c["q"])
        k.copy_(c["k"])
        c2 = dict(c, q=q, k=k)
        a, b = _check(c2)
        assert a.is_contiguous() and b.is_contiguous()
        _check_grad(c2)
    with pytest.raises(ValueError, match="neighbours"):
        _forward(dict(c, q=torch.randn(256, 50, device="cuda").bfloat16().t()))
    with pytest.raises(ValueError, match="apart"):
        _forward(dict(c, q=torch.randn(1, 256, device="cuda").bfloat16().expand(50, 256)))


def test_in_place_and_given_outputs():
    c = _case(90, 4, 2, 64, "bf16", "layer", (10, 20), True, False, seed=1)
    q, k = _forward(c)
    q1, k1 = c["q"].clone(), c["k"].clone()
    a, b = tla.qk_norm_rope(q1, k1, 4, 2, q_w=c["q_w"], q_b=c["q_b"], k_w=c["k_w"], k_b=c["k_b"], **c["rest"], q_out=q1, k_out=k1)
    assert a is q1 and b is k1 and torch.equal(q1, q) and torch.equal(k1, k)
    got = _grad(c)
    dq, dk = c["dq"].clone(), c["dk"].clone()
    out = got._replace(**{x: torch.empty_like(v) for x, v in got._asdict().items()})._replace(dq=dq, dk=dk)
    tla.qk_norm_rope_grad(c["q"], c["k"], dq, dk, 4, 2, q_w=c["q_w"], k_w=c["k_w"], bias=True, **c["rest"], out=out)
    assert all(torch.equal(x, y) for x, y in zip(got, out))
    for name in tla.QkNormRopeGrads._fields:
        one = tla.QkNormRopeGrads(**{name: torch.empty_like(getattr(got, name))})
        _grad(c, out=one)
        assert torch.equal(getattr(one, name), getattr(got, name)), name


def test_far_positions():
    # positions to the ends of int32: angles of 2 billion radians, right to fp32
    c = _case(200, 2, 2, 64, "f32", "none", (16, 16), True, False, seed=2, far=2 ** 31 - 1)
    c["rest"]["base"] = 1.0  # every pair turns a radian a step
    c["rest"]["pos"][0] = torch.tensor([-2 ** 31, 2 ** 31 - 1], dtype=torch.int32)
    # 2^31 radians are 3.4e8 turns in 64 bits: off by 2^31 2^-53 turns = 1.5e-6 u of a turn more
    _check(c)
    _check_grad(c)


def test_short_and_empty_heads():
    c = _case(20, 2, 2, 64, "f32", "l2", (16, 16), True, False, seed=3)
    c["q"][3] = 0.0
    c["q"][4] *= 1e-20  # below eps with the eps given here
    c["rest"]["eps"] = 1e-6
    q, _ = _check(c)
    assert (q[3] == 0).all()
    _check_grad(c)
    c = _case(20, 2, 2, 64, "f32", "layer", (), True, False, seed=3)
    c["q"][3] = 0.0
    c["q"][4] = 2.5
    _check(c)


def test_large_and_non_finite_heads_stay_alone():
    c = _case(20, 4, 4, 64, "f32", "rms", (16, 16), True, False, seed=4)
    q, k = _forward(c)
    g = _grad(c)
    c["q"][7, 64:128] = float("nan")
    c["q"][8, 70] = float("inf")
    c["dq"][9, 3] = float("nan")
    q2, k2 = _forward(c)
    g2 = _grad(c)
    bad = torch.zeros_like(q, dtype=torch.bool)
    bad[7:9, 64:128] = True
    assert torch.equal(q[~bad], q2[~bad]) and torch.equal(k, k2) and torch.isnan(q2[7, 64:128]).all()
    bad[9, :64] = True
    assert torch.equal(g.dq[~bad], g2.dq[~bad]) and torch.equal(g.dk, g2.dk)


def test_no_tokens():
    c = _case(0, 2, 2, 64, "bf16", "rms", (16, 16), True, False)
    q, k = _forward(c)
    assert q.shape == (0, 128) and k.shape == (0, 128)
    got = _grad(c)
    assert (got.dq_w == 0).all() and (got.dk_w == 0).all() and got.dq.shape == (0, 128)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_tokens(dtype):
    # more tokens than waves: 9000 tokens against the same call on its parts
    c = _case(9000, 3, 1, 64, dtype, "rms", (10, 10, 10), True, False, seed=5)
    q, k = _forward(c)
    for lo in range(0, 9000, 4000):
        s = slice(lo, lo + 4000)
        part = dict(c, q=c["q"][s], k=c["k"][s], rest=dict(c["rest"], pos=c["rest"]["pos"][s].contiguous()))
        q1, k1 = _forward(part)
        assert torch.equal(q[s], q1) and torch.equal(k[s], k1)
    # sums: a lane adds up to 3 tokens x 1 head group; the rest as above
    _check_grad(c)


def test_streams_graphs_and_same_bits():
    c = _case(500, 4, 2, 64, "bf16", "layer", (16, 16), True, False, seed=6)
    want, wg = _forward(c), _grad(c)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        a, g1 = _forward(c), _grad(c)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip((*want, *wg), (*a, *g1)))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a, g1 = _forward(c), _grad(c)
    for _ in range(3):
        c["q"].copy_(torch.randn_like(c["q"]))
        c["dk"].copy_(torch.randn_like(c["dk"]))
        g.replay()
        torch.cuda.synchronize()
        want, wg = _forward(c), _grad(c)
        assert all(torch.equal(x, y) for x, y in zip((*want, *wg), (*a, *g1)))


def test_more_than_2_31_values():
    n = 2_100_000
    q = torch.randn(n, 1024, device="cuda", dtype=torch.bfloat16)
    pos = torch.arange(n, device="cuda", dtype=torch.int32)[:, None].contiguous()
    a, _ = tla.qk_norm_rope(q, None, 16, pos=pos, sections=(32,))
    b, _ = tla.qk_norm_rope(q[-5:].contiguous(), None, 16, pos=pos[-5:].contiguous(), sections=(32,))
    assert n * 1024 > 2 ** 31 and torch.equal(a[-5:], b)
    g = tla.qk_norm_rope_grad(q, None, q, None, 16, pos=pos, sections=(32,))
    h = tla.qk_norm_rope_grad(q[-5:].contiguous(), None, q[-5:].contiguous(), None, 16, pos=pos[-5:].contiguous(), sections=(32,))
    assert torch.equal(g.dq[-5:], h.dq)


def test_prepared_queries_into_the_layer_and_the_delta_rule():
    # as they are used together: a view's projections, normed and rotated, through the write and read of the layer and
    # through the delta rule, and back again
    c = _case(2 * 1374, 4, 4, 64, "bf16", "l2", (16, 16), True, False, seed=7)
    q, k = _check(c)
    g = torch.Generator("cuda").manual_seed(0)
    v = torch.nn.functional.normalize(torch.randn(2 * 1374, 4, 64, generator=g, device="cuda"), dim=-1).flatten(1).bfloat16()
    theta = 0.02 * torch.randn(4, 3 * 64 * 128, generator=g, device="cuda")
    tla.ttt_write(k, v, theta, 0.1, 1, 4)
    assert torch.isfinite(tla.ttt_read(q, theta, 4)).all()
    beta = torch.rand(2 * 1374, 4, generator=g, device="cuda")
    o, state = tla.gated_delta(q, k, v, None, beta, 4)
    # what the state holds of the last tokens' values: after a full step onto a key, reading it returns its value
    one = torch.ones(1, 4, device="cuda")
    tla.gated_delta_step(q[-1:], k[-1:], v[-1:], None, one, 4, state)
    back = tla.gated_delta_step(k[-1:], k[-1:], v[-1:], None, 0 * one, 4, state)
    # k as stored in bf16 has length 1 + 2^-9: the read is off by the length's square, 2^-8, and a rounding
    assert torch.allclose(back.float(), v[-1:].float(), rtol=2.0 ** -6, atol=2.0 ** -8)
    d = tla.gated_delta_grad(q, k, v, None, beta, o, 4)
    e = tla.qk_norm_rope_grad(c["q"], c["k"], d.dq, d.dk, 4, 4, **c["rest"])
    assert torch.isfinite(e.dq).all() and torch.isfinite(e.dk).all()
    # an L2 norm's gradient has nothing along its input
    along = (e.dq.float().view(-1, 4, 64) * c["q"].float().view(-1, 4, 64)).sum(-1)
    size = e.dq.float().view(-1, 4, 64).norm(dim=-1) * c["q"].float().view(-1, 4, 64).norm(dim=-1)
    assert (along.abs() <= 2.0 ** -7 * size).all()
