"""Refusals of the 4-bit operators, on the host: bad shapes, types, pointers and workspaces never reach a launch."""
import ctypes

import pytest
import torch

import test_layer_amd as tla
from test_layer_amd import _lib

P = [ctypes.c_void_p(0x10000000 * (i + 1)) for i in range(12)]  # 16-byte aligned, 256 MB apart, never read


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def test_sizes(lib):
    assert lib.vggt3_mx4_codes_bytes(3, 1) == 3 * 64 and lib.vggt3_mx4_scales_bytes(3, 1) == 64 * 4
    assert lib.vggt3_mx4_codes_bytes(65, 129) == 65 * 128 and lib.vggt3_mx4_scales_bytes(65, 129) == 128 * 8
    assert lib.vggt3_mx4_codes_bytes(0, 128) == 0 and lib.vggt3_mx4_codes_bytes(-1, 128) == 0
    assert lib.vggt3_mx4_codes_bytes(1, 0) == 0 and lib.vggt3_mx4_codes_bytes(1, (1 << 20) + 1) == 0


def test_quantize_refusals(lib):
    def call(X=P[0], t=0, codes=P[1], scales=P[2], rows=64, k=128, dt=tla.BF16):
        return lib.vggt3_mx4_quantize(X, t, codes, scales, rows, k, dt, None)

    assert call(rows=0) == tla.OK and call(rows=0, X=None, codes=None, scales=None) == tla.OK
    assert call(rows=-1) == tla.EINVAL and call(k=0) == tla.EINVAL and call(dt=2) == tla.EINVAL
    assert call(k=(1 << 20) + 1) == tla.EUNSUPPORTED and call(rows=1 << 41) == tla.EUNSUPPORTED
    assert call(rows=1 << 39, k=128) == tla.EUNSUPPORTED  # more workgroups than one launch takes
    for who in ("X", "codes", "scales"):
        assert call(**{who: None}) == tla.EINVAL
        assert call(**{who: ctypes.c_void_p(0x10000008)}) == tla.EINVAL
    assert call(codes=P[0]) == tla.EINVAL and "overlap" in lib.vggt3_last_error().decode()
    assert call(scales=P[1]) == tla.EINVAL


def test_dequantize_refusals(lib):
    def call(codes=P[0], scales=P[1], X=P[2], rows=64, k=128, dt=tla.F32):
        return lib.vggt3_mx4_dequantize(codes, scales, X, rows, k, dt, None)

    assert call(rows=0) == tla.OK
    assert call(dt=7) == tla.EINVAL and call(rows=-5) == tla.EINVAL and call(k=-1) == tla.EINVAL
    assert call(X=None) == tla.EINVAL and call(X=P[0]) == tla.EINVAL and call(scales=ctypes.c_void_p(8)) == tla.EINVAL


def test_matmul_refusals(lib):
    ws = lib.vggt3_mx4_matmul_workspace_bytes(100, 64, 256, tla.BF16)
    assert ws > 0
    assert lib.vggt3_mx4_matmul_workspace_bytes(100, 64, 256, 5) == 0
    assert lib.vggt3_mx4_matmul_workspace_bytes(0, 64, 256, tla.BF16) == 0
    # 4-bit operands and a few tokens need none
    assert lib.vggt3_mx4_matmul_workspace_bytes(100, 64, 256, tla.MX4) == 0
    assert lib.vggt3_mx4_matmul_workspace_bytes(1, 64, 256, tla.BF16) == 0

    def call(A=P[0], As=None, at=tla.BF16, W=P[1], Ws=P[2], C=P[3], m=100, n=64, k=256, dt=tla.BF16, w=P[4], nb=1 << 20):
        return lib.vggt3_mx4_matmul(A, As, at, W, Ws, C, m, n, k, dt, w, nb, None)

    assert call(m=0) == tla.OK
    assert call(at=9) == tla.EINVAL and call(dt=tla.MX4) == tla.EINVAL
    assert call(m=-1) == tla.EINVAL and call(n=0) == tla.EINVAL and call(k=0) == tla.EINVAL
    assert call(n=(1 << 20) + 1) == tla.EUNSUPPORTED and call(m=1 << 40, n=1 << 20) == tla.EUNSUPPORTED
    assert call(As=P[5]) == tla.EINVAL  # scales beside unquantised tokens
    assert call(at=tla.MX4, As=None) == tla.EINVAL
    assert call(w=None) == tla.EWORKSPACE and call(nb=ws - 1) == tla.EWORKSPACE
    for who in ("A", "W", "Ws", "C"):
        assert call(**{who: None}) == tla.EINVAL
        assert call(**{who: ctypes.c_void_p(0x10000004)}) == tla.EINVAL
    assert call(C=P[0]) == tla.EINVAL and call(w=P[3]) == tla.EINVAL and call(w=P[1]) == tla.EINVAL


def test_freeze_and_read_refusals(lib):
    def freeze(theta=P[0], parts=P[1:7], H=1, d=1024, m=4096):
        return lib.vggt3_ttt_freeze_mx4(theta, *parts, H, d, m, None)

    assert freeze(d=64, m=128) == tla.EUNSUPPORTED and freeze(H=2) == tla.EUNSUPPORTED and freeze(d=0) == tla.EINVAL
    assert freeze(theta=None) == tla.EINVAL and freeze(parts=[P[1], P[2], P[1], P[4], P[5], P[6]]) == tla.EINVAL

    need = lib.vggt3_ttt_read_mx4_workspace_bytes(100, 1, 1024, 4096, tla.BF16)
    assert need > lib.vggt3_ttt_read_mx4_workspace_bytes(100, 1, 1024, 4096, tla.MX4) > 0
    assert lib.vggt3_ttt_read_mx4_workspace_bytes(10, 1, 1024, 4096, tla.F32) == 0

    def read(Q=P[0], Qs=None, qt=tla.BF16, parts=P[1:7], O=P[7], n=100, H=1, d=1024, m=4096, w=P[8], nb=1 << 28):
        return lib.vggt3_ttt_read_mx4(Q, Qs, qt, *parts, O, n, H, d, m, w, nb, None)

    assert read(n=0) == tla.OK
    assert read(n=-1) == tla.EINVAL and read(H=16, d=64, m=128) == tla.EUNSUPPORTED and read(qt=tla.F32) == tla.EUNSUPPORTED
    assert read(w=None) == tla.EWORKSPACE and read(nb=need - 1) == tla.EWORKSPACE
    assert read(Qs=P[9]) == tla.EINVAL and read(qt=tla.MX4) == tla.EINVAL
    assert read(O=P[0]) == tla.EINVAL and read(O=P[3]) == tla.EINVAL and read(O=P[8]) == tla.EINVAL


def test_binding_refusals():
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="GPU"):
        tla.mx4_quantize(x)
    with pytest.raises(TypeError):
        tla.mx4_quantize(x.half())
    with pytest.raises(ValueError):
        tla.mx4_quantize(x[0])
    with pytest.raises(ValueError, match="columns"):
        tla.mx4_quantize(x[:, :0])
    codes, scales = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(1, 1, 64, 4, dtype=torch.uint8)
    a = tla.Mx4(codes, scales, 64)
    with pytest.raises(ValueError, match="GPU"):
        tla.mx4_dequantize(a)
    with pytest.raises(ValueError, match="expected"):
        tla.mx4_dequantize(a._replace(k=129))
    with pytest.raises(TypeError, match="uint8"):
        tla.mx4_dequantize(a._replace(codes=codes.int()))
    with pytest.raises(TypeError):
        tla.mx4_dequantize(a, torch.float16)
    with pytest.raises(TypeError, match="Mx4"):
        tla.mx4_matmul(a, x)
    with pytest.raises(ValueError):
        tla.mx4_matmul(torch.zeros(4, 32), a)
    with pytest.raises(ValueError):
        tla.mx4_matmul(a, a, out=torch.zeros(4, 5))
    with pytest.raises(TypeError, match="FrozenMx4"):
        tla.ttt_read_mx4(x.bfloat16(), (a, a, a))
    with pytest.raises(ValueError):
        tla.mx4_quantize(x, out=a._replace(k=63))


def test_matrices_of_more_tiles_than_a_launch_takes(lib):
    # a launch has fewer than 2^32 threads in all: 2^24 workgroups of 256, one a scale tile of 64 x 128
    most = ((1 << 24) - 1) * 64
    assert lib.vggt3_mx4_scales_bytes(most, 1) == most * 4 and lib.vggt3_mx4_scales_bytes(most + 1, 1) == 0
    two = ((1 << 23) - 1) * 64  # rows of two tiles
    assert lib.vggt3_mx4_codes_bytes(two, 256) == two * 128 and lib.vggt3_mx4_codes_bytes(two + 1, 129) == 0
    far = [ctypes.c_void_p(1 << 44), ctypes.c_void_p(1 << 45), ctypes.c_void_p(1 << 46)]
    assert lib.vggt3_mx4_quantize(far[0], 0, far[1], far[2], most + 1, 1, tla.BF16, None) == tla.EUNSUPPORTED
    assert lib.vggt3_mx4_dequantize(far[0], far[1], far[2], most + 1, 1, tla.BF16, None) == tla.EUNSUPPORTED
    assert lib.vggt3_mx4_matmul_workspace_bytes(most + 1, 1, 1, tla.BF16) == 0


@pytest.mark.parametrize("k", [2 ** 31, 2 ** 32 + 64])
def test_widths_that_do_not_fit_32_bits(k):
    # the C calls take widths as int32, where 2^32 + 64 would pass as 64 and leave the rest of the result unwritten
    x = torch.empty((2, k), dtype=torch.bfloat16, device="meta")
    with pytest.raises(ValueError, match="columns"):
        tla.mx4_quantize(x)
    with pytest.raises(ValueError, match="columns"):
        tla.mx4_quantize(x.t(), transpose=True)
    kp = (k + 127) // 128 * 128
    a = tla.Mx4(torch.empty((2, kp // 2), dtype=torch.uint8, device="meta"),
                torch.empty((1, kp // 128, 64, 4), dtype=torch.uint8, device="meta"), k)
    with pytest.raises(ValueError, match="columns"):
        tla.mx4_dequantize(a)
    with pytest.raises(ValueError, match="columns"):
        tla.mx4_matmul(a, a)
    with pytest.raises(ValueError, match="columns"):
        tla.block_join(x, x, pre="rms")
    with pytest.raises(ValueError, match="columns"):
        tla.block_join_grad(x, x, x, x, pre="rms")
