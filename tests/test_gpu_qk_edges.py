"""The query/key preparation and its gradient where values are not finite and where positions are far, on the GPU."""
import math
import random
from decimal import Context, Decimal, localcontext

import pytest
import torch

import test_layer_amd as tla

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
# heads by 4 pairs apart, by neighbours, handed over through LDS and value by value, of each number of lanes
SHAPES = [(64, (16, 16), False), (64, (), False), (64, (32,), True), (64, (12, 10, 10), False), (63, (10, 7), False), (128, (32, 16), False),
          (104, (20, 6), False), (200, (40, 20), True), (512, (100,), False), (7, (2,), True)]


def _randn(*shape, seed=0, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def _pos(n, sections, far=1000):
    if not sections:
        return None
    return torch.randint(-far, far, (n, len(sections)), generator=torch.Generator().manual_seed(3), dtype=torch.int32).cuda()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,sections,interleaved", SHAPES, ids=str)
def test_length_of_a_head_with_nan(d, sections, interleaved, dtype):
    # |x| is NaN, and so are x / max(|x|, eps) and its gradient, all over the head and nowhere else
    n, heads = 9, 3
    x, dy = (_randn(n, heads * d, seed=s, dtype=DT[dtype]) for s in (1, 2))
    rest = dict(norm="l2", eps=1e-6, pos=_pos(n, sections), sections=sections, interleaved=interleaved)
    y, _ = tla.qk_norm_rope(x, None, heads, **rest)
    g = tla.qk_norm_rope_grad(x, None, dy, None, heads, **rest).dq
    for row, head, at in ((0, 0, 0), (4, 2, d - 1), (8, 1, d // 2)):
        bad = x.clone()
        bad[row, head * d + at] = float("nan")
        spoilt = torch.zeros_like(x, dtype=torch.bool)
        spoilt[row, head * d:head * d + d] = True
        for got, want in ((tla.qk_norm_rope(bad, None, heads, **rest)[0], y),
                          (tla.qk_norm_rope_grad(bad, None, dy, None, heads, **rest).dq, g)):
            assert torch.isnan(got[spoilt]).all() and torch.equal(got[~spoilt], want[~spoilt])


def _partners(d, sections, interleaved):
    """The channels that each channel's result is made of, axis by axis (per_axis)."""
    of = {ch: {ch} for ch in range(d)}
    off = 0
    for c in sections:
        for j in range(c):
            a, b = (off + 2 * j, off + 2 * j + 1) if interleaved else (off + j, off + j + c)
            of[a] = of[b] = {a, b}
        off += 2 * c
    return of


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,sections,interleaved", [s for s in SHAPES if s[1]], ids=str)
def test_channels_that_are_not_rotated_are_their_own(d, sections, interleaved, dtype):
    # no norm: a value that is not finite spoils its pair's channels, and of channels that are not rotated itself alone
    n = 5
    x, dy = (_randn(n, d, seed=s, dtype=DT[dtype]) for s in (4, 5))
    rest = dict(norm=None, pos=_pos(n, sections) * 2 + 1, sections=sections, interleaved=interleaved)
    y, _ = tla.qk_norm_rope(x, None, 1, **rest)
    g = tla.qk_norm_rope_grad(x, None, dy, None, 1, **rest).dq
    of = _partners(d, sections, interleaved)
    for ch in range(d):
        bad_x, bad_dy = x.clone(), dy.clone()
        bad_x[2, ch], bad_dy[2, ch] = float("inf"), float("nan")
        mine = torch.tensor([ch in of[c] for c in range(d)]).cuda()
        for got, want in ((tla.qk_norm_rope(bad_x, None, 1, **rest)[0], y),
                          (tla.qk_norm_rope_grad(x, None, bad_dy, None, 1, **rest).dq, g)):
            assert torch.equal(got[2, ~mine], want[2, ~mine]) and not torch.isfinite(got[2, mine]).any(), ch
            assert torch.equal(got[[0, 1, 3, 4]], want[[0, 1, 3, 4]])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 63, 128, 104, 200, 7])
def test_norms_alone_leave_channels_to_themselves(d, dtype):
    # no rotation: an infinite value is NaN after an L2 norm, and the others 0; an infinite weight or bias is its own channel's
    n = 5
    x = _randn(n, d, seed=6, dtype=DT[dtype])
    w, b = _randn(d, seed=7), _randn(d, seed=8)
    rest = dict(norm="rms", eps=1e-6)
    y, _ = tla.qk_norm_rope(x, None, 1, q_w=w, q_b=b, **rest)
    for ch in range(d):
        bad = x.clone()
        bad[1, ch] = float("inf")
        got, _ = tla.qk_norm_rope(bad, None, 1, norm="l2")
        others = torch.arange(d, device="cuda") != ch
        assert torch.isnan(got[1, ch]) and (got[1, others] == 0).all()
        for name in ("q_w", "q_b"):
            v = dict(q_w=w.clone(), q_b=b.clone())
            v[name][ch] = float("inf")
            got, _ = tla.qk_norm_rope(x, None, 1, **v, **rest)
            assert torch.equal(got[:, others], y[:, others]) and torch.isinf(got[:, ch]).all()


TURN = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


def _turns(base, j, size):
    """Turns a position step of pair j, to 60 digits."""
    with localcontext(Context(prec=60)):
        return (-Decimal(base).ln() * j / size).exp() / TURN


@pytest.mark.parametrize("base", [1.0, 50.0, 100.0, 10000.0, 0.5])
@pytest.mark.parametrize("d,sections,per_axis", [(64, (16, 16), True), (64, (12, 10, 10), True), (128, (40, 24), False), (512, (256,), True)],
                         ids=str)
def test_angles_of_far_positions(d, sections, per_axis, base):
    # a rotated (1, 0) is (cos, sin) of the angle. Reduced to a part of a turn, that is rounded once to fp32 (2 pi 2^-26 =
    # 1.6 u), sine and cosine by u each and the product with 1 not at all: 4 u, at any position. (Those taken here are the
    # ones of many where one double's rounding of the pairs' turns shows most.)
    axes = len(sections)
    r = random.Random(d + axes)
    rows = [[-2 ** 31] * axes, [2 ** 31 - 1] * axes]
    sizes = [c if per_axis else sum(sections) for c in sections]
    before = [0 if per_axis else sum(sections[:a]) for a in range(axes)]
    turns = [[_turns(base, before[a] + j, sizes[a]) for j in range(c)] for a, c in enumerate(sections)]

    def worst(t, count):
        seen = [r.randrange(2 ** 30, 2 ** 31) * r.choice((1, -1)) for _ in range(count)]
        return max(seen, key=lambda p: abs(Decimal(float(t) * p) - t * p))

    with localcontext(Context(prec=60)):
        for i in range(60):
            rows.append([worst(turns[a][i % min(c, 6)], 50) for a, c in enumerate(sections)])
        for i in range(20):
            rows.append([r.randrange(-2 ** (i + 11), 2 ** (i + 11)) for _ in sections])
        want_cos, want_sin = [], []
        for row in rows:
            t = [(p * x) % 1 for p, ts in zip(row, turns) for x in ts]
            want_cos.append([math.cos(float(x * TURN)) for x in t])
            want_sin.append([math.sin(float(x * TURN)) for x in t])
    n, pairs = len(rows), sum(sections)
    x = torch.zeros(n, d)
    x[:, 0:2 * pairs:2] = 1.0
    x = x.cuda()
    rest = dict(norm=None, pos=torch.tensor(rows, dtype=torch.int32).cuda(), sections=sections, base=base, per_axis=per_axis,
                interleaved=True)
    y = tla.qk_norm_rope(x, None, 1, **rest)[0].double().cpu()[:, :2 * pairs]
    g = tla.qk_norm_rope_grad(x, None, x, None, 1, **rest).dq.double().cpu()[:, :2 * pairs]
    cos, sin = torch.tensor(want_cos, dtype=torch.float64), torch.tensor(want_sin, dtype=torch.float64)
    for got, c, s in ((y, cos, sin), (g, cos, -sin)):
        assert (got[:, 0::2] - c).abs().max() <= 4 * 2.0 ** -24
        assert (got[:, 1::2] - s).abs().max() <= 4 * 2.0 ** -24
