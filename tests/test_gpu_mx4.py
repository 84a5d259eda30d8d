"""4-bit quantisation, products and the frozen read against the float64 oracle on the GPU.

Tolerances, derived before the first run:
- Quantisation and its inverse are exact: bit for bit.
- A product adds P <= kp products of 4-bit values in fp32. Each is exact; the sums are off by at most
  P 2^-24 times the sum of magnitudes (one rounding an addition). Rounding the result adds half a step of the
  output type: 2^-8 (bf16) or 2^-24 (fp32) relative.
"""
import numpy as np
import pytest
import torch

import test_layer_amd as tla
from gpu_util import to64
from oracle import mx4

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _x(rows, k, seed, dtype, scale=1.0):
    g = np.random.default_rng(seed)
    x = g.standard_normal((rows, k)) * np.exp(g.standard_normal((rows, 1))) * scale
    x[:, g.random(k) < 0.02] *= 20
    if rows > 2:
        x[1] = 0
    return torch.tensor(x, dtype=torch.float32).to(DT[dtype]).cuda()


def _w(n, k, seed, scale=None):
    w = np.random.default_rng(seed).standard_normal((n, k)) * (k ** -0.5 if scale is None else scale)
    return torch.tensor(w, dtype=torch.float32).cuda()


def _stored(a):
    return a.codes.cpu().numpy(), a.scales.cpu().numpy()


def _vals(a):
    code, s = mx4.load(*_stored(a))
    return mx4.values(code, s, a.k)


def _check_stored(a, x64):
    want_c, want_s = mx4.store(*mx4.quantize(x64))
    codes, scales = _stored(a)
    assert np.array_equal(scales, want_s)
    assert np.array_equal(codes, want_c)


SHAPES = [(1, 1), (1, 32), (3, 31), (5, 8), (16, 33), (63, 128), (64, 129), (65, 127), (130, 1000), (257, 1024)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,k", SHAPES)
def test_quantize_bit_exact(rows, k, dtype):
    x = _x(rows, k, rows + k, dtype)
    a = tla.mx4_quantize(x)
    _check_stored(a, to64(x))
    for out in ("bf16", "f32"):
        assert np.array_equal(to64(tla.mx4_dequantize(a, DT[out])), mx4.roundtrip(to64(x)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,k", SHAPES)
def test_quantize_transposed_is_the_quantised_transpose(rows, k, dtype):
    x = _x(rows, k, rows + k + 1, dtype)
    a, b = tla.mx4_quantize(x), tla.mx4_quantize(x.t().contiguous(), transpose=True)
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_every_tie_and_range_end(dtype):
    # multiples of 1/16 up to 8 hold every grid value and midpoint; their scales run over the exponents
    base = np.arange(-128, 128) / 16.0
    rows = []
    for e in (-149, -140, -134, -130, -127, -126, -100, -3, 0, 5, 100, 124):
        rows.append(base * 2.0 ** e)
    x = torch.tensor(np.array(rows), dtype=torch.float64).to(torch.float32).to(DT[dtype]).cuda()
    a = tla.mx4_quantize(x)
    _check_stored(a, to64(x))
    for out in ("bf16", "f32"):
        assert np.array_equal(to64(tla.mx4_dequantize(a, DT[out])), mx4.roundtrip(to64(x)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_non_finite_values_make_their_block_nan(dtype):
    x = _x(70, 200, 3, dtype)
    x[2, 40], x[68, 199], x[69, 0] = float("inf"), float("nan"), float("-inf")
    a = tla.mx4_quantize(x)
    _check_stored(a, to64(x))
    got = to64(tla.mx4_dequantize(a, DT[dtype]))
    assert np.array_equal(got, mx4.roundtrip(to64(x)), equal_nan=True)
    # and its row of a product, no other
    w = _w(33, 200, 4)
    c = to64(tla.mx4_matmul(a, tla.mx4_quantize(w), torch.float32))
    bad = np.isnan(c)
    assert bad[[2, 68, 69]].all() and not np.delete(bad, [2, 68, 69], 0).any()
    w[7, 1] = float("nan")
    c = to64(tla.mx4_matmul(tla.mx4_quantize(_x(20, 200, 5, dtype)), tla.mx4_quantize(w), torch.float32))
    assert np.isnan(c[:, 7]).all() and not np.isnan(np.delete(c, 7, 1)).any()


def _check_product(c, av, wv, out):
    want = mx4.matmul(av, wv)
    mag = mx4.matmul(np.abs(av), np.abs(wv))
    kp = -(-av.shape[1] // 128) * 128
    tol = kp * 2.0 ** -24 * mag + (2.0 ** -8 if out == "bf16" else 2.0 ** -24) * np.abs(want)
    err = np.abs(to64(c) - want)
    assert (err <= tol).all(), float((err / np.maximum(tol, 1e-300)).max())


MNK = [(1, 1, 1), (1, 4096, 1024), (2, 7, 33), (5, 64, 64), (15, 130, 256), (16, 33, 384), (17, 100, 127), (33, 257, 640),
       (64, 128, 4096), (65, 999, 1000), (127, 31, 8192), (129, 129, 129), (300, 520, 512), (1000, 1024, 128),
       (1374, 48, 96), (2100, 1000, 1000)]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k", MNK)
def test_matmul(m, n, k, out):
    a, w = tla.mx4_quantize(_x(m, k, m, "bf16")), tla.mx4_quantize(_w(n, k, n))
    _check_product(tla.mx4_matmul(a, w, DT[out]), _vals(a), _vals(w), out)


def _check_product_on_gpu(m, n, k, out):
    """A product too large for numpy: float64 on the GPU, on the values the operands stand for."""
    g = torch.Generator("cuda").manual_seed(k)
    a = tla.mx4_quantize(torch.randn(m, k, generator=g, device="cuda") * torch.randn(m, 1, generator=g, device="cuda"))
    w = tla.mx4_quantize(torch.randn(n, k, generator=g, device="cuda"))
    c = tla.mx4_matmul(a, w, DT[out])
    av, wv = tla.mx4_dequantize(a, torch.float32).double(), tla.mx4_dequantize(w, torch.float32).double()
    kp = -(-k // 128) * 128
    for r in range(0, m, 8192):
        want = av[r:r + 8192] @ wv.t()
        tol = kp * 2.0 ** -24 * (av[r:r + 8192].abs() @ wv.abs().t()) + (2.0 ** -8 if out == "bf16" else 2.0 ** -24) * want.abs()
        assert bool(((c[r:r + 8192].double() - want).abs() <= tol).all()), r


# each kernel with more tiles than workgroups, ragged edges, and from one step of 128 columns on
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("k", [40, 256, 384, 500, 640, 1100])
@pytest.mark.parametrize("m,n", [(9001, 2500), (9000, 2501), (68701, 4096), (70000, 4001)])
def test_matmul_of_many_tiles(m, n, k, out):
    _check_product_on_gpu(m, n, k, out)


@pytest.mark.parametrize("m,n,k", [(11000, 1024, 4096), (22001, 1000, 2100), (300, 60000, 256), (5, 70000, 300)])
def test_matmul_of_long_sides(m, n, k):
    _check_product_on_gpu(m, n, k, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 1024, 1024), (3, 100, 1000), (8, 64, 8192), (16, 999, 1000), (17, 64, 256),
                                   (200, 300, 333)])
def test_matmul_of_tokens_is_that_of_their_4_bits(m, n, k, dtype):
    x, w = _x(m, k, 9, dtype), tla.mx4_quantize(_w(n, k, 8))
    c = tla.mx4_matmul(x, w, torch.float32)
    assert torch.equal(c, tla.mx4_matmul(tla.mx4_quantize(x), w, torch.float32))


def test_matmul_of_far_scales():
    # products whose scales multiply to the ends of fp32: exact 2^-120 and 2^120, and an overflow to Inf
    a, w = torch.zeros(3, 64, device="cuda"), torch.zeros(2, 64, device="cuda")
    a[0, 0], a[1, 0], a[2, 0] = 2.0 ** -100, 2.0 ** 100, 2.0 ** 100
    w[0, 0], w[1, 0] = 2.0 ** -20, 2.0 ** 20
    c = tla.mx4_matmul(tla.mx4_quantize(a), tla.mx4_quantize(w), torch.float32)
    assert c.tolist() == [[2.0 ** -120, 2.0 ** -80], [2.0 ** 80, 2.0 ** 120], [2.0 ** 80, 2.0 ** 120]]
    w[1, 0] = 2.0 ** 60
    assert tla.mx4_matmul(tla.mx4_quantize(a), tla.mx4_quantize(w), torch.float32)[1, 1].item() == float("inf")


def test_matmul_writes_its_rows_only():
    m, n, k = 70, 130, 200
    whole = torch.full((m * n + 64,), 7.0, device="cuda")
    tla.mx4_matmul(_x(m, k, 1, "f32"), tla.mx4_quantize(_w(n, k, 2)), torch.float32, out=whole[:m * n].view(m, n))
    assert (whole[m * n:] == 7).all()


def test_zero_rows():
    w = tla.mx4_quantize(_w(64, 128, 1))
    x = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    a = tla.mx4_quantize(x)
    assert a.codes.shape == (0, 64) and a.scales.numel() == 0
    assert tla.mx4_matmul(x, w).shape == (0, 64) and tla.mx4_matmul(a, w).shape == (0, 64)
    assert tla.mx4_dequantize(a).shape == (0, 128)


@pytest.fixture(scope="module")
def frozen():
    g = torch.Generator().manual_seed(5)
    theta = torch.randn(3 * 1024 * 4096, generator=g)
    theta[: 2 * 1024 * 4096] *= 1.5 / 32
    theta[2 * 1024 * 4096:] *= 1 / 64
    theta = theta.view(1, -1).cuda()
    return theta, tla.ttt_freeze_mx4(theta)


def test_freeze_is_the_quantised_transposes(frozen):
    theta, f = frozen
    t = theta.view(3, -1)
    for part, src in ((f.gate, t[0].view(1024, 4096)), (f.up, t[1].view(1024, 4096)), (f.down, t[2].view(4096, 1024))):
        want = tla.mx4_quantize(src.t().contiguous())
        assert torch.equal(part.codes, want.codes) and torch.equal(part.scales, want.scales)


@pytest.mark.parametrize("n", [1, 2, 16, 17, 64, 100, 257, 1374])
def test_read_frozen(frozen, n):
    _, f = frozen
    q = torch.randn(n, 1024, generator=torch.Generator().manual_seed(n)).to(torch.bfloat16).cuda()
    o = to64(tla.ttt_read_mx4(q, f))
    wg, wu, wd = _vals(f.gate), _vals(f.up), _vals(f.down)
    h = mx4.swiglu(mx4.roundtrip(to64(q)), wg, wu)
    want = mx4.matmul(mx4.roundtrip(h), wd)
    # H may land on the other side of a rounding border where it lies within 2e-5 of one (its fp32 error: 1024
    # additions 2^-24 of magnitudes that exceed the sum ~20-fold); such a value moves by one step, at most 2 scales.
    code, s = mx4.quantize(h)
    v = np.abs(h.reshape(n, 128, 32)) / np.ldexp(1.0, s.astype(np.int64) - 127)[..., None]
    mids = np.array([.25, .75, 1.25, 1.75, 2.5, 3.5, 5.0, 4.0, 8.0])
    close = (np.abs(v[..., None] - mids) <= 2e-5 * 8).any(-1)
    step = close * 2.0 * np.ldexp(1.0, s.astype(np.int64) - 127)[..., None]
    move = mx4.matmul(step.reshape(n, 4096), np.abs(wd))
    mag = mx4.matmul(np.abs(mx4.roundtrip(h)), np.abs(wd))
    tol = move + 4096 * 2.0 ** -24 * mag + 2.0 ** -8 * (np.abs(want) + move)
    assert (np.abs(o - want) <= tol).all()
    # and as a whole near the fp64 result: half a bf16 step, and few values moved
    assert np.linalg.norm(o - want) <= 2.0 ** -8 * np.linalg.norm(want)
    # tokens in 4 bits already give the same bits
    assert torch.equal(tla.ttt_read_mx4(tla.mx4_quantize(q), f).cpu(), torch.tensor(o).to(torch.bfloat16))


def test_read_of_many_tokens_agrees_with_that_of_a_few(frozen):
    # other kernels, the same numbers up to the order of fp32 sums (and an H value here and there that this moves
    # over a rounding border): far below the half step of bf16 that both are rounded by
    _, f = frozen
    q = torch.randn(9003, 1024, generator=torch.Generator().manual_seed(8)).to(torch.bfloat16).cuda()
    o = tla.ttt_read_mx4(q, f)
    for r in (0, 250, 4096, 8987):
        few = to64(tla.ttt_read_mx4(q[r:r + 16], f))
        assert np.linalg.norm(to64(o[r:r + 16]) - few) <= 2.0 ** -9 * np.linalg.norm(few), r


def test_read_chunks_agree_with_their_parts(frozen):
    _, f = frozen
    n = 131072 + 77  # one whole chunk and a short one
    q = torch.randn(n, 1024, generator=torch.Generator("cuda").manual_seed(1), device="cuda").to(torch.bfloat16)
    o = tla.ttt_read_mx4(q, f)
    assert torch.equal(o[:131072], tla.ttt_read_mx4(q[:131072], f))
    assert torch.equal(o[131072:], tla.ttt_read_mx4(q[131072:], f))
    assert torch.equal(o, tla.ttt_read_mx4(tla.mx4_quantize(q), f))
    assert torch.isfinite(o).all() and o.float().std() > 0.1


def test_read_follows_the_read_in_bf16(frozen):
    # 4 bits carry about 10 % error a value; a sum of independent errors keeps that relative size
    theta, f = frozen
    q = torch.randn(300, 1024, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    a, b = to64(tla.ttt_read_mx4(q, f)), to64(tla.ttt_read(q, theta, 1, d_hidden=4096))
    assert np.linalg.norm(a - b) / np.linalg.norm(b) < 0.5
    assert (a * b).sum() / np.linalg.norm(a) / np.linalg.norm(b) > 0.9


def test_same_bits_each_time():
    x, w = _x(333, 1000, 1, "bf16"), tla.mx4_quantize(_w(777, 1000, 2))
    c = tla.mx4_matmul(x, w)
    for _ in range(3):
        assert torch.equal(c, tla.mx4_matmul(x, w))


@pytest.mark.parametrize("m", [1, 100])
def test_other_stream_and_graph_replay(m):
    w = tla.mx4_quantize(_w(256, 512, 2))
    x = _x(m, 512, 1, "bf16")
    want = tla.mx4_matmul(x, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = tla.mx4_matmul(x, w)
    s.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(want)
    ws = torch.empty(max(1, tla.mx4_matmul_workspace_bytes(m, 256, 512, tla.BF16)), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tla.mx4_matmul(x, w, out=out, workspace=ws)
    for seed in (5, 6, 7):
        x.copy_(_x(m, 512, seed, "bf16"))
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, tla.mx4_matmul(x, w))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k", [(1, 40, 31), (2, 100, 37), (4, 64, 1001), (4, 4096, 4096), (7, 33, 129), (16, 70, 1024),
                                   (1, 17, 16384), (1, 17, 16385), (15, 16, 999)])
def test_tokens_quantised_in_the_product(m, n, k, dtype):
    x, w = _x(m, k, k, dtype), tla.mx4_quantize(_w(n, k, n))
    x[m - 1, k // 2] = float("inf")  # one block of the last row
    c = tla.mx4_matmul(x, w, torch.float32)
    want = tla.mx4_matmul(tla.mx4_quantize(x), w, torch.float32)
    assert torch.isnan(c[m - 1]).all() and torch.isnan(want[m - 1]).all()
    assert torch.equal(c[:m - 1], want[:m - 1])


def test_two_products_at_once_and_two_captured_graphs():
    w = tla.mx4_quantize(_w(1024, 1024, 2))
    xs = [_x(3000, 1024, s, "bf16") for s in (1, 2)]
    want = [tla.mx4_matmul(x, w) for x in xs]
    outs, graphs = [torch.empty_like(c) for c in want], []
    need = tla.mx4_matmul_workspace_bytes(3000, 1024, 1024, tla.BF16)
    for x, out in zip(xs, outs):
        g, ws = torch.cuda.CUDAGraph(), torch.empty(need, dtype=torch.uint8, device="cuda")
        with torch.cuda.graph(g):
            tla.mx4_matmul(x, w, out=out, workspace=ws)
        graphs.append((g, ws))
    for _ in range(3):
        for out in outs:
            out.zero_()
        torch.cuda.synchronize()
        for g, _ in graphs:
            with torch.cuda.stream(torch.cuda.Stream()):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, c) for o, c in zip(outs, want))


@pytest.mark.parametrize("n", [5, 40, 200, 700])
def test_read_where_gate_times_up_passes_fp32(n):
    # Unit 5: gate = -2^40 q0, up = 2^40 q0. q0 = 2^35 in one row, so gate * up is past fp32 there, but silu(gate) * up
    # is 0, as in the other rows (q0 = 1): the same bits as with up = 0. By 16 rows, by 64 rows, by 64 x 64 tiles and
    # by 256 x 256 tiles, from tokens and from 4 bits.
    g = torch.Generator().manual_seed(n)
    theta = torch.randn(3, 1024 * 4096, generator=g) / 32
    gate, up = theta[0].view(1024, 4096), theta[1].view(1024, 4096)
    gate[0], up[0] = 0.0, 0.0
    gate[0, 5] = -2.0 ** 40
    zero = tla.ttt_freeze_mx4(theta.view(1, -1).cuda())
    up[0, 5] = 2.0 ** 40
    f = tla.ttt_freeze_mx4(theta.view(1, -1).cuda())
    q = torch.randn(n, 1024, generator=g)
    q[:, 0] = 1.0
    q[3, 0] = 2.0 ** 35
    q = q.to(torch.bfloat16).cuda()
    o = tla.ttt_read_mx4(q, f)
    assert torch.isfinite(o).all()
    assert torch.equal(o, tla.ttt_read_mx4(q, zero))
    assert torch.equal(o, tla.ttt_read_mx4(tla.mx4_quantize(q), f))


def test_more_than_2_31_values():
    rows, k, n = 2_200_001, 1024, 1000
    g = torch.Generator("cuda").manual_seed(6)
    x = torch.randn(rows, k, generator=g, device="cuda", dtype=torch.bfloat16)
    a = tla.mx4_quantize(x)
    at = rows // 64 * 64 - 640  # a whole scale tile's first row
    few = tla.mx4_quantize(x[at:].clone())
    assert torch.equal(a.codes[at:], few.codes) and torch.equal(a.scales[at // 64:], few.scales)
    back = tla.mx4_dequantize(a)
    assert torch.equal(back[at:], tla.mx4_dequantize(few))
    w = tla.mx4_quantize(torch.randn(n, k, generator=g, device="cuda"))
    c = tla.mx4_matmul(a, w)  # 2.2e9 values
    want = back[at:].double() @ tla.mx4_dequantize(w, torch.float32).double().t()
    mag = back[at:].double().abs() @ tla.mx4_dequantize(w, torch.float32).double().abs().t()
    assert bool(((c[at:].double() - want).abs() <= k * 2.0 ** -24 * mag + 2.0 ** -8 * want.abs()).all())


@pytest.mark.parametrize("m,n,k", [(3, 20, 1 << 20), (40, 100, (1 << 20) - 5), (1100, 1100, 1 << 18), (70, 1 << 20, 200),
                                   (1, 1 << 20, 33)])
def test_matmul_of_the_longest_sides(m, n, k):
    _check_product_on_gpu(m, n, k, "f32")


@pytest.mark.parametrize("n", [5, 40, 200, 700])
def test_read_of_a_non_finite_token_leaves_the_others(frozen, n):
    _, f = frozen
    q = torch.randn(n, 1024, generator=torch.Generator().manual_seed(n)).to(torch.bfloat16).cuda()
    want = tla.ttt_read_mx4(q, f)
    q[3, 1000], q[n - 2, 0] = float("nan"), float("-inf")
    for o in (tla.ttt_read_mx4(q, f), tla.ttt_read_mx4(tla.mx4_quantize(q), f)):
        assert torch.isnan(o[[3, n - 2]]).all()
        o[[3, n - 2]] = want[[3, n - 2]]
        assert torch.equal(o, want)


@pytest.mark.parametrize("n", [1, 100, 700])
def test_read_on_another_stream_and_in_graphs(frozen, n):
    # quantise, read and quantise back as one captured pass, replayed on new tokens between eager passes
    _, f = frozen
    q = torch.randn(n, 1024, generator=torch.Generator().manual_seed(n)).to(torch.bfloat16).cuda()

    def both(a, o, back, ws):
        tla.mx4_quantize(q, out=a)
        tla.ttt_read_mx4(a, f, out=o, workspace=ws)
        tla.mx4_dequantize(a, out=back)

    def fresh():
        return (tla.mx4_quantize(torch.zeros_like(q)), torch.empty_like(q), torch.empty_like(q),
                torch.empty(tla.read_mx4_workspace_bytes(n, 1024, 4096, tla.MX4), dtype=torch.uint8, device="cuda"))

    eager, other, caught = fresh(), fresh(), fresh()
    both(*eager)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        both(*other)
    s.synchronize()
    assert torch.equal(other[1], eager[1]) and torch.equal(other[2], eager[2])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both(*caught)
    for seed in (1, 2, 3):
        q.copy_(torch.randn(n, 1024, generator=torch.Generator().manual_seed(seed)))
        caught[1].zero_()
        g.replay()
        torch.cuda.synchronize()
        both(*eager)
        assert torch.equal(caught[1], eager[1]) and torch.equal(caught[2], eager[2])
        assert torch.equal(caught[0].codes, eager[0].codes) and torch.equal(caught[0].scales, eager[0].scales)
