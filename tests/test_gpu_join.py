"""Block join and its gradient against the float64 oracle on the GPU.

Tolerances, derived before the first run, in u = 2^-24 (an fp32 rounding) and half a step of the output type
(2^-8 relative for bf16, u for fp32):
- A row sum adds at most 16 values a thread, 6 butterfly steps and 8 waves: 30 roundings, so a mean is off by
  30 u mean|v| and, with the few operations round it, a norm by 40 u (|v| + mean|v|) rstd |w|.
- A gradient row goes through two such sums one after the other (80 u), and the norm after the block through two
  more (160 u); sums over tokens add at most (rows a unit + 4 + blocks / 16 + 4) < 60 roundings at these sizes.
  All are bounded by 256 u times the same formula with every term's magnitude in place of the term.
"""
import numpy as np
import pytest
import torch

import test_layer_amd as tla
from gpu_util import to64
from oracle import join, mx4

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def _case(n, C, dtype, post, pre, gate, per, scale, bias, seed=0):
    g = np.random.default_rng(seed)

    def t(*shape, std=1.0, mean=0.0, dt=torch.float32):
        return torch.tensor(g.standard_normal(shape) * std + mean, dtype=torch.float32).to(dt).cuda()

    dt = DT[dtype]
    c = dict(x=t(n, C, std=1.5, dt=dt), f=t(n, C, std=0.7, mean=0.3, dt=dt), post=post, pre=pre, per=per,
             gate=t(-(-n // per), C, std=0.5, mean=1.0, dt=dt) if gate else None, scale=t(C, std=0.2, mean=0.3) if scale else None,
             post_w=t(C, std=0.2, mean=1.0) if post != "none" else None, pre_w=t(C, std=0.2, mean=1.0) if pre != "none" else None,
             post_b=t(C, std=0.3) if post != "none" and bias else None, pre_b=t(C, std=0.3) if pre != "none" and bias else None,
             dr=t(n, C, dt=dt), dy=t(n, C, dt=dt) if pre != "none" else None)
    return c


def _o(c, *names):
    return [None if c[k] is None else to64(c[k]) for k in names]


def _args(c):
    return dict(gate=c["gate"], gate_tokens=c["per"], scale=c["scale"], post=c["post"], post_w=c["post_w"], post_b=c["post_b"],
                pre=c["pre"], pre_w=c["pre_w"])


def _norm_mag(v, kind, w, b):
    """Magnitude of a norm's terms: |w| rstd (|v| + mean|v|) + |b|, and rstd."""
    if kind == "none":
        return np.abs(v)
    rstd = join.norm(v, kind)[2]
    m = rstd * (np.abs(v) + np.abs(v).mean(1, keepdims=True)) * (1.0 if w is None else np.abs(w))
    return m if b is None else m + np.abs(b)


def _check_forward(c, dtype, mx=False):
    r, y = tla.block_join(c["x"], c["f"], pre_b=c["pre_b"], mx4=mx, **_args(c))
    x, f, gate, scale, pw, pb, w, b = _o(c, "x", "f", "gate", "scale", "post_w", "post_b", "pre_w", "pre_b")
    want = join.join(x, f, gate, c["per"], scale, c["post"], pw, pb)
    sg = np.abs((1.0 if scale is None else scale) * join.spread(gate, c["per"], len(x)))
    tol = 40 * U * (sg * _norm_mag(f, c["post"], pw, pb) + np.abs(x)) + HALF[dtype] * np.abs(want)
    assert (np.abs(to64(r) - want) <= tol).all()
    if c["pre"] == "none":
        assert y is None
        return r, y
    r64 = to64(r)  # the norm is that of the stored stream
    want = join.norm(r64, c["pre"], w, b)[0]
    if not mx:
        tol = 40 * U * _norm_mag(r64, c["pre"], w, b) + HALF[dtype] * np.abs(want)
        assert (np.abs(to64(y) - want) <= tol).all()
    return r, y


MODES = [("none", "none", False, 1, True, False), ("none", "rms", True, 1, False, False), ("rms", "none", True, 3, True, True),
         ("layer", "layer", True, 7, True, True), ("rms", "rms", False, 1, True, False), ("none", "layer", False, 1, False, True),
         ("layer", "rms", True, 1000, False, False), ("layer", "layer", True, 1, True, False)]
SHAPES = [(1, 1), (1, 1024), (2, 33), (5, 64), (37, 100), (64, 512), (65, 513), (130, 1024), (40, 1025), (23, 2048), (9, 4096),
          (6, 5000), (3, 8192), (700, 24), (33, 128), (21, 256),
          (19, 200), (50, 7), (31, 515), (12, 1999), (5, 4095), (3, 8191)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("mode", MODES, ids=lambda m: "-".join(map(str, m)))
@pytest.mark.parametrize("n,C", SHAPES)
def test_forward(n, C, mode, dtype):
    post, pre, gate, per, scale, bias = mode
    _check_forward(_case(n, C, dtype, post, pre, gate, per, scale, bias, n + C), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,C", SHAPES)
def test_y_in_4_bits_is_y_quantised(n, C, dtype):
    c = _case(n, C, dtype, "rms", "layer", True, 2, True, True, n)
    if n > 3:
        c["x"][2, C // 2] = float("nan")
    r, y = tla.block_join(c["x"], c["f"], pre_b=c["pre_b"], **_args(c))
    r4, y4 = tla.block_join(c["x"], c["f"], pre_b=c["pre_b"], mx4=True, **_args(c))
    want = tla.mx4_quantize(y)
    assert torch.equal(r.view(torch.int16), r4.view(torch.int16))
    assert torch.equal(y4.codes, want.codes) and torch.equal(y4.scales, want.scales)


@pytest.mark.parametrize("pre", ["rms", "layer"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_alone(pre, dtype):
    c = _case(50, 200, dtype, "none", pre, False, 1, False, True)
    r, y = tla.block_join(c["x"], pre=pre, pre_w=c["pre_w"], pre_b=c["pre_b"])
    assert r is None
    x, w, b = _o(c, "x", "pre_w", "pre_b")
    want = join.norm(x, pre, w, b)[0]
    assert (np.abs(to64(y) - want) <= 40 * U * _norm_mag(x, pre, w, b) + HALF[dtype] * np.abs(want)).all()
    # and it is the y of a join that gives the same stream
    zero = torch.zeros_like(c["x"])
    r2, y2 = tla.block_join(c["x"], zero, pre=pre, pre_w=c["pre_w"], pre_b=c["pre_b"])
    assert torch.equal(r2, c["x"]) and torch.equal(y2, y)


def test_in_place_and_given_outputs():
    c = _case(300, 1024, "bf16", "layer", "rms", True, 50, True, True)
    r, y = tla.block_join(c["x"], c["f"], pre_b=c["pre_b"], **_args(c))
    x, y2 = c["x"].clone(), torch.empty_like(y)
    r3, y3 = tla.block_join(x, c["f"], pre_b=c["pre_b"], r=x, y=y2, **_args(c))
    assert r3 is x and y3 is y2 and torch.equal(x, r) and torch.equal(y2, y)
    got = tla.block_join_grad(r, c["f"], c["dr"], c["dy"], pre_bias=True, **_args(c))
    dr = c["dr"].clone()
    out = got._replace(**{k: torch.empty_like(v) for k, v in got._asdict().items()})._replace(dx=dr)
    tla.block_join_grad(r, c["f"], dr, c["dy"], out=out, **_args(c))
    for k, v in got._asdict().items():
        assert torch.equal(getattr(out, k), v), k


def test_rows_far_from_zero_mean_and_constant_rows():
    # a mean 1000 times the deviation: the two-pass variance keeps its digits; a constant row has deviation 0
    x = torch.randn(20, 512, generator=torch.Generator().manual_seed(0)) + 1000
    x[3] = 5.0
    x[4] = 0.0
    x = x.cuda()
    _, y = tla.block_join(x, pre="layer")
    want = join.norm(to64(x), "layer")[0]
    # the centred values are off by 40 u (|v| + mean|v|) = 80 u 1000, over a deviation of 1 (or sqrt(eps))
    rstd = join.norm(to64(x), "layer")[2]
    assert (np.abs(to64(y) - want) <= 80 * U * np.abs(to64(x)) * rstd + 40 * U * np.abs(want)).all()
    assert (to64(y)[4] == 0).all()


def test_non_finite_rows_stay_alone():
    c = _case(9, 256, "f32", "layer", "rms", True, 1, True, True)
    c["f"][2, 5] = float("inf")
    c["x"][7, 0] = float("nan")
    r, y = tla.block_join(c["x"], c["f"], pre_b=c["pre_b"], **_args(c))
    bad = torch.isnan(y).all(1)
    assert bad.tolist() == [i in (2, 7) for i in range(9)]
    assert torch.isfinite(r[[0, 1, 3, 4, 5, 6, 8]]).all() and torch.isfinite(y[~bad]).all()


def _magnitudes(c):
    """join.grads with every term's magnitude in place of the term."""
    r, f, dr, dy, gate, scale, pw, pb, w = _o(c, "x", "f", "dr", "dy", "gate", "scale", "post_w", "post_b", "pre_w")
    n, C = r.shape

    def hat_mag(v, kind):
        return np.abs(v) if kind == "none" else _norm_mag(v, kind, None, None)

    def back_mag(d, v, kind):
        if kind == "none":
            return d
        h, rstd = hat_mag(v, kind), join.norm(v, kind)[2]
        return rstd * (d + h * (d * h).mean(1, keepdims=True) + d.mean(1, keepdims=True))

    out = {}
    d = np.abs(dr)
    if c["pre"] != "none":
        h = hat_mag(r, c["pre"])
        out["dpre_w"], out["dpre_b"] = (np.abs(dy) * h).sum(0), np.abs(dy).sum(0)
        d = d + back_mag(np.abs(dy) * np.abs(w), r, c["pre"])
    out["dx"] = d
    h = _norm_mag(f, c["post"], pw, pb)
    g, s = np.abs(join.spread(gate, c["per"], n)), 1.0 if scale is None else np.abs(scale)
    out["dscale"] = (d * g * h).sum(0)
    per = min(c["per"], n)
    groups = -(-n // per)
    p = np.zeros((groups * per, C))
    p[:n] = d * s * h
    out["dgate"] = p.reshape(groups, per, C).sum(1)
    dh = d * g * s
    out["dpost_w"], out["dpost_b"] = (dh * hat_mag(f, c["post"])).sum(0), dh.sum(0)
    out["df"] = back_mag(dh * (1.0 if pw is None else np.abs(pw)), f, c["post"])
    return out


def _check_grad(c, dtype):
    got = tla.block_join_grad(c["x"], c["f"], c["dr"], c["dy"], pre_bias=c["pre_b"] is not None, **_args(c))
    r, f, dr, dy, gate, scale, pw, pb, w = _o(c, "x", "f", "dr", "dy", "gate", "scale", "post_w", "post_b", "pre_w")
    want = join.grads(r, f, dr, dy, gate, c["per"], scale, c["post"], pw, pb, c["pre"], w)
    mag = _magnitudes(c)
    given = {"dx": True, "df": True, "dgate": c["gate"], "dscale": c["scale"], "dpost_w": c["post_w"], "dpost_b": c["post_b"],
             "dpre_w": c["pre_w"], "dpre_b": c["pre_b"]}
    for k, v in got._asdict().items():
        assert (v is None) == (given[k] is None), k
        if v is None:
            continue
        half = HALF[dtype] if k in ("dx", "df", "dgate") else U
        err = np.abs(to64(v) - want[k])
        tol = 256 * U * mag[k] + half * np.abs(want[k])
        assert (err <= tol).all(), (k, float((err / np.maximum(tol, 1e-300)).max()))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("mode", MODES, ids=lambda m: "-".join(map(str, m)))
@pytest.mark.parametrize("n,C", SHAPES)
def test_grad(n, C, mode, dtype):
    post, pre, gate, per, scale, bias = mode
    _check_grad(_case(n, C, dtype, post, pre, gate, per, scale, bias, n + C), dtype)


@pytest.mark.parametrize("per", [1, 2, 3, 50, 137, 1374, 2999, 3000, 10 ** 6, 2 ** 32, 2 ** 63 - 1])
def test_gate_groups_across_units(per):
    # groups inside a unit's rows, ending with them, spanning two and many, and one longer than the tokens
    c = _case(3000, 40, "f32", "rms", "layer", True, per, True, True, per % 1000)
    _check_forward(c, "f32")
    _check_grad(c, "f32")


def test_grad_at_more_rows_than_one_a_unit():
    c = _case(20011, 1024, "bf16", "layer", "layer", True, 1374, True, True)
    got = tla.block_join_grad(c["x"], c["f"], c["dr"], c["dy"], pre_bias=True, **_args(c))
    again = tla.block_join_grad(c["x"], c["f"], c["dr"], c["dy"], pre_bias=True, **_args(c))
    r, f, dr, dy, gate, scale, pw, pb, w = _o(c, "x", "f", "dr", "dy", "gate", "scale", "post_w", "post_b", "pre_w")
    want = join.grads(r, f, dr, dy, gate, 1374, scale, "layer", pw, pb, "layer", w)
    for k, v in got._asdict().items():
        assert torch.equal(v, getattr(again, k)), k
        half = 2.0 ** -8 if k in ("dx", "df", "dgate") else U
        e = np.linalg.norm(to64(v) - want[k]) / np.linalg.norm(want[k])
        assert e <= half + 256 * U, (k, e)


def test_grad_of_the_norm_alone():
    c = _case(77, 300, "f32", "none", "layer", False, 1, False, True)
    got = tla.block_join_grad(c["x"], dy=c["dy"], pre="layer", pre_w=c["pre_w"], pre_bias=True)
    r, dy, w = _o(c, "x", "dy", "pre_w")
    want = join.grads(r, None, None, dy, pre="layer", pre_w=w)
    zero = dict(c, dr=torch.zeros_like(c["dr"]))
    mag = _magnitudes(zero)
    assert got.df is None and got.dscale is None and got.dgate is None
    for k in ("dx", "dpre_w", "dpre_b"):
        assert (np.abs(to64(getattr(got, k)) - want[k]) <= 256 * U * mag[k] + U * np.abs(want[k])).all(), k


def test_unwanted_gradients_are_left_alone():
    c = _case(60, 128, "f32", "rms", "rms", True, 4, True, False)
    full = tla.block_join_grad(c["x"], c["f"], c["dr"], c["dy"], **_args(c))
    only = tla.block_join_grad(c["x"], c["f"], c["dr"], c["dy"], out=tla.BlockJoinGrads(df=torch.empty_like(c["f"])), **_args(c))
    assert torch.equal(only.df, full.df) and only.dx is None and only.dgate is None and only.dscale is None


def test_no_tokens():
    x = torch.empty(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    r, y = tla.block_join(x, x.clone(), pre="rms", pre_w=w)
    assert r.shape == y.shape == (0, 64)
    _, y4 = tla.block_join(x, x.clone(), pre="rms", pre_w=w, mx4=True)
    assert y4.codes.shape == (0, 64)
    got = tla.block_join_grad(x, x.clone(), x.clone(), x.clone(), pre="rms", pre_w=w, scale=w)
    assert got.dx.shape == (0, 64) and (got.dscale == 0).all() and (got.dpre_w == 0).all()


def test_streams_and_graph_replay():
    c = _case(500, 1024, "bf16", "layer", "layer", True, 100, True, True)

    def both(**kw):
        return (tla.block_join(c["x"], c["f"], pre_b=c["pre_b"], **_args(c), **{k: v for k, v in kw.items() if k in "ry"}),
                tla.block_join_grad(c["x"], c["f"], c["dr"], c["dy"], pre_bias=True, **_args(c),
                                    **{k: v for k, v in kw.items() if k not in "ry"}))

    (r, y), grads = both()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        (r2, y2), grads2 = both()
    s.synchronize()
    assert torch.equal(r, r2) and torch.equal(y, y2) and all(torch.equal(a, b) for a, b in zip(grads, grads2))
    ws = torch.empty(tla.block_join_grad_workspace_bytes(500, 1024, tla.BF16), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both(r=r2, y=y2, out=grads2, workspace=ws)
    for seed in (1, 2, 3):
        new = _case(500, 1024, "bf16", "layer", "layer", True, 100, True, True, seed)
        for k in ("x", "f", "gate", "dr", "dy", "scale", "post_w"):
            c[k].copy_(new[k])
        for t in (r2, y2, *grads2):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        (r, y), grads = both()
        assert torch.equal(r, r2) and torch.equal(y, y2) and all(torch.equal(a, b) for a, b in zip(grads, grads2))


def test_block_on_frozen_weights_end_to_end():
    """The operators as a served block uses them: norm -> 4 bits -> frozen MLP -> join -> norm -> 4 bits -> product."""
    n, per = 300, 100
    g = torch.Generator().manual_seed(2)
    theta = torch.randn(1, 3 * 1024 * 4096, generator=g) / 32
    c = _case(n, 1024, "bf16", "layer", "rms", True, per, True, True)
    frozen = tla.ttt_freeze_mx4(theta.cuda())
    head = tla.mx4_quantize((torch.randn(77, 1024, generator=g) / 32).cuda())
    _, q = tla.block_join(c["x"], pre="layer", mx4=True)
    o = tla.ttt_read_mx4(q, frozen)
    r, y = tla.block_join(c["x"], o, pre_b=c["pre_b"], mx4=True, **_args(c))
    z = tla.mx4_matmul(y, head, torch.float32)
    # each step against the oracle on the step's own inputs
    qv = to64(tla.mx4_dequantize(q, torch.float32))
    plain = to64(tla.block_join(c["x"], pre="layer")[1])
    assert np.array_equal(qv, mx4.roundtrip(plain))
    assert torch.equal(o, tla.ttt_read_mx4(torch.tensor(plain).to(torch.bfloat16).cuda(), frozen))
    _check_forward(dict(c, f=o), "bf16", mx=True)
    yv, hv = to64(tla.mx4_dequantize(y, torch.float32)), to64(tla.mx4_dequantize(head, torch.float32))
    assert (np.abs(to64(z) - yv @ hv.T) <= 1024 * U * (np.abs(yv) @ np.abs(hv).T)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,C,per", [(1000, 300, 5), (1001, 130, 20), (1374, 1024, 30), (3000, 257, 40), (2999, 512, 47),
                                     (2999, 512, 49)])
def test_gate_groups_of_a_few_units(n, C, per, dtype):
    # groups that 2 to 17 units share, the last one short
    _check_grad(_case(n, C, dtype, "layer", "rms", True, per, True, True, per), dtype)


@pytest.mark.parametrize("C", [1, 33, 99, 127, 129, 500, 999, 2050])
def test_odd_rows_in_4_bits_on_two_streams_at_once(C):
    # a row of odd width ends inside a unit's columns; two calls on streams of their own, outputs of their own
    a, b = (_case(301, C, d, "rms", "layer", True, 7, True, True, C + i) for i, d in enumerate(("bf16", "f32")))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    torch.cuda.synchronize()
    for c, s in zip((a, b), streams):
        with torch.cuda.stream(s):
            got.append(tla.block_join(c["x"], c["f"], pre_b=c["pre_b"], mx4=True, **_args(c)))
    torch.cuda.synchronize()
    for c, (r, y4) in zip((a, b), got):
        r1, y1 = tla.block_join(c["x"], c["f"], pre_b=c["pre_b"], **_args(c))
        assert torch.equal(r, r1)
        want = tla.mx4_quantize(y1)
        assert torch.equal(y4.codes, want.codes) and torch.equal(y4.scales, want.scales)


# -------------------------------------------------------------------------------------- many rows a unit of threads
# The kernels' units take one row each up to 524,288 / threads rows (forward) and 256 (gradient), and a range of rows
# beyond. The shapes below give 2 or more rows a unit to each unit size (forward: 16, 64, 128, 256, 512 threads;
# gradient: 16, 32, 64, 128, 256, 512 and 512 x 16 values), with rows of whole pieces and of odd width.

LONG_FORWARD = [(70001, 40), (66001, 99), (65600, 128), (66001, 200), (20011, 500), (20011, 1024), (17003, 999), (9001, 2048),
                (9001, 1999), (4500, 4096), (4201, 4095), (2500, 5000), (2500, 8191), (2101, 8192)]


@pytest.mark.parametrize("per,dtype", [(1, "bf16"), (3, "f32"), (1009, "bf16"), (1009, "f32")])
@pytest.mark.parametrize("n,C", LONG_FORWARD)
def test_forward_of_many_rows_a_unit_is_that_of_slices(n, C, per, dtype):
    # Slices small enough for one row a unit, with the gate's rows repeated for their tokens: the same arithmetic on
    # each row, so the same bits. In place too, and into 4 bits, whose last scale tile is cut.
    g = torch.Generator("cuda").manual_seed(n + per)

    def t(*shape, std=1.0, mean=0.0, dt=torch.float32):
        return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dt)

    dt = DT[dtype]
    x, f, gate = t(n, C, std=1.5, dt=dt), t(n, C, std=0.7, mean=0.3, dt=dt), t(-(-n // per), C, std=0.5, mean=1.0, dt=dt)
    kw = dict(scale=t(C, std=0.2, mean=0.3), post="rms", post_w=t(C, std=0.2, mean=1.0), post_b=t(C, std=0.3), pre="layer",
              pre_w=t(C, std=0.2, mean=1.0), pre_b=t(C, std=0.3))
    r, y = tla.block_join(x, f, gate, per, **kw)
    r4, y4 = tla.block_join(x, f, gate, per, mx4=True, **kw)
    assert torch.equal(r4, r)
    want = tla.mx4_quantize(y)
    assert torch.equal(y4.codes, want.codes) and torch.equal(y4.scales, want.scales)
    threads = 16 if C <= 256 else 64 if C <= 1024 else 128 if C <= 2048 else 256 if C <= 4096 else 512
    step = 524288 // threads
    assert n > step
    rows = gate if per == 1 else gate.repeat_interleave(per, 0)[:n]
    for a in range(0, n, step):
        s = slice(a, min(n, a + step))
        r1, y1 = tla.block_join(x[s].clone(), f[s].clone(), rows[s].clone(), 1, **kw)
        assert torch.equal(r[s], r1) and torch.equal(y[s], y1), a
    r5, y5 = tla.block_join(x, f, gate, per, r=x, **kw)
    assert r5 is x and torch.equal(x, r) and torch.equal(y5, y)


@pytest.mark.parametrize("post,pre", [("none", "none"), ("layer", "rms"), ("none", "layer")])
@pytest.mark.parametrize("n,C,dtype", [(33000, 24, "bf16"), (33001, 99, "f32"), (9000, 999, "bf16"), (8300, 1024, "f32"),
                                       (4200, 2048, "bf16"), (2100, 4100, "f32")])
def test_forward_of_many_rows_a_unit(n, C, dtype, post, pre):
    _check_forward(_case(n, C, dtype, post, pre, post == "layer", 250, True, post != "none", n), dtype)


# A channel sum adds the rows of a unit (at most 14 here), the up to 16 units of a workgroup, the workgroups' parts in
# 64 runs of at most 23 and then 6 levels of a tree: at most 14 + 15 + 23 + 6 roundings. A shared gate group adds its
# rows in a unit, then at most 16 units in turn, or its units in 16 runs and 4 levels: fewer. With the 160 of a row that
# the head of this file counts, all stay below the 256 u of _check_grad.
@pytest.mark.parametrize("n,C,dtype", [(40000, 40, "bf16"), (33001, 99, "f32"), (20000, 200, "f32"), (20001, 257, "bf16"),
                                       (9000, 500, "bf16"), (5000, 1024, "f32"), (6000, 999, "bf16"), (2600, 2048, "bf16"),
                                       (1500, 1999, "f32"), (900, 4096, "bf16"), (900, 4095, "f32"), (1100, 5000, "bf16"),
                                       (900, 8192, "bf16"), (900, 8192, "f32"), (600, 8191, "f32"), (900, 8191, "bf16")])
@pytest.mark.parametrize("per", [1, 3, 400])
def test_grad_of_many_rows_a_unit(n, C, dtype, per):
    _check_grad(_case(n, C, dtype, "layer", "rms" if per % 2 else "layer", True, per, True, True, n + per), dtype)


@pytest.mark.parametrize("post,pre", [("none", "rms"), ("rms", "none"), ("rms", "rms")])
@pytest.mark.parametrize("n,C,dtype", [(9000, 40, "f32"), (2000, 1024, "bf16"), (1500, 2048, "f32"), (700, 6000, "bf16")])
def test_grad_of_many_rows_a_unit_without_a_shared_gate(n, C, dtype, post, pre):
    _check_grad(_case(n, C, dtype, post, pre, False, 1, post == "rms", False, n), dtype)


def test_grad_of_a_scene_value_by_value():
    _check_grad(_case(20011, 1024, "bf16", "layer", "layer", True, 1374, True, True), "bf16")


# ------------------------------------------------------------------------------------------------- values past fp32

@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("C", [64, 99])
def test_infinite_scale_without_a_bias(C, post):
    # scale = Inf: r = x + Inf h, an Inf of h's sign; the other channels as they were
    c = _case(30, C, "f32", post, "none", True, 1, True, False)
    r, _ = tla.block_join(c["x"], c["f"], **_args(c))
    h = to64(r) - to64(c["x"])
    c["scale"][3] = float("inf")
    got = to64(tla.block_join(c["x"], c["f"], **_args(c))[0])
    assert np.array_equal(got[:, 3], np.sign(h[:, 3]) * np.inf)
    assert np.array_equal(np.delete(got, 3, 1), np.delete(to64(r), 3, 1))


@pytest.mark.parametrize("post", ["none", "rms"])
def test_infinite_gradient_without_a_bias(post):
    # dr = Inf at one token and channel: dscale there is an Inf of h's sign
    c = _case(30, 64, "f32", post, "none", False, 1, True, False)
    c["dr"][5, 3] = float("inf")
    got = tla.block_join_grad(c["x"], c["f"], c["dr"], **_args(c))
    f = to64(c["f"])
    h = join.norm(f, post, None if c["post_w"] is None else to64(c["post_w"]))[0]
    assert got.dscale[3].item() == np.sign(h[5, 3]) * np.inf
    assert torch.isfinite(got.dscale[:3]).all() and torch.isfinite(got.dscale[4:]).all()


def test_zeros_of_no_tokens_whatever_the_weights():
    x, w = torch.empty(0, 64, device="cuda"), torch.full((64,), float("inf"), device="cuda")
    got = tla.block_join_grad(x, x.clone(), x.clone(), x.clone(), post="rms", post_w=w, post_b=w.clone(), pre="rms",
                              pre_w=w.clone(), scale=w.clone())
    assert all((v == 0).all() for v in (got.dscale, got.dpost_w, got.dpost_b, got.dpre_w))


# ------------------------------------------------------------------------------------------ calls that are left over

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("C", [40, 99, 1024])
def test_vectors_left_out_and_their_gradients(C, kind, dtype):
    # no weights, no scale, biases alone; their gradients asked for all the same, those of the rest not
    n, per = 77, 5
    c = _case(n, C, dtype, kind, kind, True, per, False, True, C)
    c["post_w"] = c["pre_w"] = None
    _check_forward(c, dtype)
    f32 = [torch.full((C,), 7.0, device="cuda") for _ in range(5)]
    out = tla.BlockJoinGrads(None, torch.empty_like(c["f"]), None, *f32)
    got = tla.block_join_grad(c["x"], c["f"], c["dr"], c["dy"], out=out, **_args(c))
    assert got is out
    ones = dict(c, post_w=torch.ones(C, device="cuda"), pre_w=torch.ones(C, device="cuda"), scale=torch.ones(C, device="cuda"))
    want = tla.block_join_grad(c["x"], c["f"], c["dr"], c["dy"], pre_bias=True, **_args(ones))
    for k in ("df", "dscale", "dpost_w", "dpost_b", "dpre_w", "dpre_b"):
        assert torch.equal(getattr(got, k), getattr(want, k)), k
    _check_grad(ones, dtype)


@pytest.mark.parametrize("n,C", [(1, 40), (500, 99), (1000, 1024), (300, 5000)])
def test_grad_without_dr_is_that_of_zeros(n, C):
    c = _case(n, C, "bf16", "layer", "rms", True, 3, True, False, n)
    want = tla.block_join_grad(c["x"], c["f"], torch.zeros_like(c["dr"]), c["dy"], **_args(c))
    got = tla.block_join_grad(c["x"], c["f"], None, c["dy"], **_args(c))
    for k, v in want._asdict().items():
        assert (v is None) == (getattr(got, k) is None) and (v is None or torch.equal(getattr(got, k), v)), k


def test_more_than_2_31_values():
    n, C, per = 2_200_001, 1024, 1374
    g = torch.Generator("cuda").manual_seed(3)
    x, f, dr, dy = (torch.randn(n, C, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(4))
    gate = torch.randn(-(-n // per), C, generator=g, device="cuda", dtype=torch.bfloat16)
    kw = dict(scale=torch.randn(C, generator=g, device="cuda"), post="rms", pre="layer")
    r, y = tla.block_join(x, f, gate, per, **kw)
    y4 = tla.block_join(x, f, gate, per, mx4=True, **kw)[1]
    got = tla.block_join_grad(r, f, dr, dy, gate, per, pre_bias=True, **kw)
    rows = n // 64 * 64 - 640  # a whole scale tile's first row
    own = gate[torch.arange(rows, n, device="cuda") // per].contiguous()
    s = slice(rows, n)
    tail = [t[s].clone() for t in (x, f, dr, dy)]
    r1, y1 = tla.block_join(*tail[:2], own, 1, **kw)
    assert torch.equal(r[s], r1) and torch.equal(y[s], y1)
    want = tla.mx4_quantize(y1)
    assert torch.equal(y4.codes[s], want.codes) and torch.equal(y4.scales[rows // 64:], want.scales)
    few = tla.block_join_grad(r1, *tail[1:], own, 1, **kw)
    assert torch.equal(got.dx[s], few.dx) and torch.equal(got.df[s], few.df)
    # sum of dy: at most 1433 rows in a unit, 23 + 6 joins
    total, mag = torch.zeros(C, dtype=torch.float64, device="cuda"), torch.zeros(C, dtype=torch.float64, device="cuda")
    for part in dy.split(200_000):
        total += part.double().sum(0)
        mag += part.double().abs().sum(0)
    assert bool(((got.dpre_b.double() - total).abs() <= 1500 * U * mag).all())
