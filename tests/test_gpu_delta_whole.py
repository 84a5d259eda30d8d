"""The gated delta rule's bf16 outputs where large terms nearly cancel: every product takes its fp32 operands whole.

Inputs are made so that each result is the difference of two neighbouring 24-bit values below 2, with all other terms 0,
and known in closed form. Tolerance, derived before the first run, in u = 2^-24: at most 4 of a sum's additions round (the
others add zeros), each by u of the partial sum, |a| + |b| < 4 here: 16 u = 2^-20; and half a step of bf16 (2^-8 relative)
of the result. (Operands cut to 16 bits would be off by up to 2^-17.)
"""
import pytest
import torch

import test_layer_amd as tla

pytestmark = pytest.mark.gpu
DIMS = [(64, 64), (128, 64), (64, 128), (128, 128)]
BF = torch.bfloat16


def _neighbours(shape, seed):
    """Pairs of 24-bit values in (1, 2), 1 to 200 steps apart."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randint(256, 2 ** 23, shape, generator=g).double()
    m = torch.randint(1, 201, shape, generator=g).double()
    return ((2 ** 23 + x) / 2 ** 23).float().cuda(), ((2 ** 23 + x - m) / 2 ** 23).float().cuda()


def _near(got, want):
    assert got.dtype == BF
    err = (got.double() - want).abs()
    assert (err <= 2.0 ** -20 + 2.0 ** -8 * want.abs()).all(), float((err - 2.0 ** -8 * want.abs()).max() * 2 ** 20)


def _hot(n, heads, d, *entries):
    """[n, heads, d] of zeros with (channel of each row, value) set."""
    x = torch.zeros(n, heads, d, dtype=BF, device="cuda")
    for at, value in entries:
        x[torch.arange(n, device="cuda"), :, at.cuda()] = value
    return x


# one chunk and a short one; pieces; enough chunks x heads for waves of 64 columns
@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("n,heads", [(40, 2), (700, 1), (33000, 16)])
def test_reads_of_nearly_equal_rows(n, heads, dk, dv):
    # no keys: o = S^T q of the first state, q = its row 2i minus row 2i + 1
    a, b = _neighbours((1, heads, dk // 2, dv), 1)
    state = torch.stack([a, b], 3).reshape(1, heads, dk, dv)
    i = torch.arange(n) % (dk // 2)
    q = _hot(n, heads, dk, (2 * i, 1.0), (2 * i + 1, -1.0)).flatten(1)
    v = torch.ones(n, heads * dv, dtype=BF, device="cuda")
    o, last = tla.gated_delta(q, torch.zeros_like(q), v, None, torch.ones(n, heads, device="cuda"), heads, state=state)
    want = (a.double() - b.double())[0, :, i.cuda()].transpose(0, 1).flatten(1)
    _near(o, want)
    assert torch.equal(last, state)


@pytest.mark.parametrize("dk,dv", DIMS)
def test_reads_of_nearly_equal_steps(dk, dv):
    # keys of one channel each: u = beta, and o_t is the difference of two tokens' steps, of this chunk and of the one before
    n, heads = 64, 3
    t = torch.arange(n)
    a, b = _neighbours((n // 2, heads), 2)
    beta = torch.stack([a / 2, b / 2], 1).reshape(n, heads)
    first = torch.where(t % 2 == 1, t - 1, (t - 2).clamp(min=0))
    first = torch.where((t >= 32) & (t % 4 < 2), t - t % 2 - 32, first)
    q = _hot(n, heads, dk, (first, 1.0), (first + 1, -1.0))
    q[0] = 0
    o, _ = tla.gated_delta(q.flatten(1), _hot(n, heads, dk, (t, 1.0)).flatten(1), torch.ones(n, heads * dv, dtype=BF, device="cuda"),
                           None, beta, heads)
    want = beta.double()[first] - beta.double()[first + 1]
    want[0] = 0
    _near(o.view(n, heads, dv), want[..., None].expand(n, heads, dv))


@pytest.mark.parametrize("dk,dv", DIMS)
def test_reads_of_nearly_equal_decays(dk, dv):
    # o_t = D_{t, t-1} - D_{t, t-2}, whose exps are off by 2 u each and whose exponents by 1 u: within the 16 u
    n, heads = 64, 2
    t = torch.arange(n)
    g = torch.rand(n, heads, generator=torch.Generator().manual_seed(3)) * -0.3
    g[1::2] *= 2.0 ** -14
    q = _hot(n, heads, dk, ((t - 1).clamp(min=0), 1.0), ((t - 2).clamp(min=0), -1.0))
    q[:2] = 0
    o, _ = tla.gated_delta(q.flatten(1), _hot(n, heads, dk, (t, 1.0)).flatten(1), torch.ones(n, heads * dv, dtype=BF, device="cuda"),
                           g.cuda(), torch.ones(n, heads, device="cuda"), heads)
    want = torch.zeros(n, heads, dtype=torch.float64)
    want[2:] = g[2:].double().exp() * -torch.expm1(g[1:-1].double())
    _near(o.view(n, heads, dv), want.cuda()[..., None].expand(n, heads, dv))
