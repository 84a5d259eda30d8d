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


@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("n,heads", [(40, 2), (700, 1), (33000, 16)])
def test_gradients_by_nearly_equal_columns(n, heads, dk, dv):
    # no keys: dq = S dO and dk = dS u, with dO and u = v a column 2i minus column 2i + 1
    (a, b), (c, d) = (_neighbours((1, heads, dk, dv // 2), s) for s in (4, 5))
    state, dstate = (torch.stack(x, 4).reshape(1, heads, dk, dv) for x in ((a, b), (c, d)))
    i = torch.arange(n) % (dv // 2)
    v = _hot(n, heads, dv, (2 * i, 1.0), (2 * i + 1, -1.0)).flatten(1)
    none = torch.zeros(n, heads * dk, dtype=BF, device="cuda")
    got = tla.gated_delta_grad(none, none, v, None, torch.ones(n, heads, device="cuda"), v, heads, dstate=dstate, state=state)
    at = i.cuda()
    _near(got.dq, (a.double() - b.double())[0, :, :, at].permute(2, 0, 1).flatten(1))
    _near(got.dk, (c.double() - d.double())[0, :, :, at].permute(2, 0, 1).flatten(1))


@pytest.mark.parametrize("dk,dv", DIMS)
def test_key_gradients_by_nearly_equal_reads(dk, dv):
    # one token a sequence, key and query of channel 0, whose state is 0: dR = dO, so dk = -S dO and dq = S dO
    heads, n = 2, dv // 2
    a, b = _neighbours((n, heads, dk, dv // 2), 6)
    a[:, :, 0] = b[:, :, 0] = 0
    state = torch.stack([a, b], 4).reshape(n, heads, dk, dv)
    i = torch.arange(n)
    k = _hot(n, heads, dk, (0 * i, 1.0)).flatten(1)
    do = _hot(n, heads, dv, (2 * i, 1.0), (2 * i + 1, -1.0)).flatten(1)
    got = tla.gated_delta_grad(k, k.clone(), torch.zeros_like(do), None, torch.ones(n, heads, device="cuda"), do, heads, state=state,
                               cu_seqlens=torch.arange(n + 1, dtype=torch.int32, device="cuda"), max_seqlen=1)
    at = i.cuda()
    want = (a.double() - b.double())[at, :, :, at].flatten(1)
    _near(got.dq, want)
    _near(got.dk, -want)


@pytest.mark.parametrize("dk,dv", DIMS)
def test_gradients_by_nearly_equal_tokens(dk, dv):
    # three tokens in turn: key e_i with u = beta; key -e_i with u = beta + delta (a full step on v = delta, of which the
    # first left -beta); a key and query of its own with dO = one channel, whose F and E with the two before, and with all
    # pairs before these, are beta and beta + delta: dq = -delta at their channels, dk = delta
    turns, heads = 30, 2
    n = 3 * turns
    a, b = _neighbours((turns, heads), 7)
    beta = torch.ones(n, heads, device="cuda")
    beta[0::3] = b / 2
    delta = (a - b) / 2  # 1 to 200 times 2^-24: values of bf16 too
    v = torch.zeros(n, heads, dv, dtype=BF, device="cuda")
    v[0::3] = 1.0
    v[1::3] = delta.to(BF)[..., None]
    i = torch.arange(turns)
    k = torch.zeros(n, heads, dk, dtype=BF, device="cuda")
    k[0::3], k[1::3] = _hot(turns, heads, dk, (i, 1.0)), _hot(turns, heads, dk, (i, -1.0))
    q = torch.zeros_like(k)
    q[2::3] = k[2::3] = _hot(turns, heads, dk, (dk - 1 - i, 1.0))
    do = torch.zeros_like(v)
    do[2::3] = _hot(turns, heads, dv, (i, 1.0))
    got = tla.gated_delta_grad(q.flatten(1), k.flatten(1), v.flatten(1), None, beta, do.flatten(1), heads)
    want = torch.zeros(turns, heads, dk, dtype=torch.float64, device="cuda")
    want[:, :, :turns] = delta.double().T[None] * (i[None, :] <= i[:, None]).cuda()[:, None]
    _near(got.dq.view(n, heads, dk)[2::3], -want)
    _near(got.dk.view(n, heads, dk)[2::3], want)


@pytest.mark.parametrize("dk,dv", DIMS)
def test_gradients_by_nearly_equal_queries(dk, dv):
    # no keys: dk = F^T q, the last two tokens' queries e_0 and -e_0 and their F beta and (1 + 2^-15) beta
    n, heads = 64, 2
    b = _neighbours((n, heads), 8)[0] / 2
    v = torch.ones(n, heads, dv, dtype=BF, device="cuda")
    v[..., 1] = 2.0 ** -8 + 2.0 ** -15
    q, do = torch.zeros(n, heads, dk, dtype=BF, device="cuda"), torch.zeros_like(v)
    q[n - 2, :, 0], q[n - 1, :, 0] = 1.0, -1.0
    do[n - 2:, :, 0] = torch.tensor([1.0, 1 - 2.0 ** -8], dtype=BF, device="cuda")[:, None]
    do[n - 1, :, 1] = 1.0
    got = tla.gated_delta_grad(q.flatten(1), torch.zeros_like(q).flatten(1), v.flatten(1), None, b, do.flatten(1), heads)
    want = torch.zeros(n, heads, dk, dtype=torch.float64, device="cuda")
    want[:, :, 0] = -b.double() * 2.0 ** -15
    want[n - 1, :, 0] -= b[n - 1].double()
    _near(got.dk.view(n, heads, dk), want)
