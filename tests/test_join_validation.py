"""Refusals of the block join and its gradient, on the host."""
import ctypes

import pytest
import torch

import test_layer_amd as tla
from test_layer_amd import _lib

P = [ctypes.c_void_p(0x10000000 * (i + 1)) for i in range(24)]


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def _join(lib, **kw):
    a = dict(x=P[0], f=P[1], gate=P[2], per=1, scale=P[3], post=1, post_w=P[4], post_b=P[5], pre=2, pre_w=P[6], pre_b=P[7],
             eps=1e-6, r=P[8], y=P[9], yc=None, ys=None, n=10, C=64, dt=tla.BF16)
    a.update(kw)
    return lib.vggt3_block_join(a["x"], a["f"], a["gate"], a["per"], a["scale"], a["post"], a["post_w"], a["post_b"], a["pre"],
                                a["pre_w"], a["pre_b"], a["eps"], a["r"], a["y"], a["yc"], a["ys"], a["n"], a["C"], a["dt"],
                                None)


def test_join_refusals(lib):
    def call(**kw):
        return _join(lib, **kw)

    assert call(n=0) == tla.OK
    assert call(dt=2) == tla.EINVAL and call(n=-1) == tla.EINVAL and call(C=0) == tla.EINVAL
    assert call(C=8193) == tla.EUNSUPPORTED and call(n=(1 << 31) + 1) == tla.EUNSUPPORTED
    assert call(post=3) == tla.EINVAL and call(pre=-1) == tla.EINVAL
    assert call(eps=-1.0) == tla.EINVAL and call(eps=float("nan")) == tla.EINVAL and call(eps=float("inf")) == tla.EINVAL
    assert call(per=0) == tla.EINVAL
    assert call(post=0) == tla.EINVAL  # a weight without its norm
    assert call(pre=0) == tla.EINVAL and call(pre=0, pre_w=None, pre_b=None) == tla.EINVAL  # y without a norm
    assert call(f=None) == tla.EINVAL
    bare = dict(f=None, gate=None, scale=None, post=0, post_w=None, post_b=None)
    assert call(**bare) == tla.EINVAL  # r without f
    assert call(**bare, r=None, pre=0, pre_w=None, pre_b=None, y=None) == tla.EINVAL  # nothing to do
    assert call(y=None) == tla.EINVAL and call(yc=P[10], ys=P[11]) == tla.EINVAL  # no y, or two
    assert call(y=None, yc=P[10]) == tla.EINVAL
    assert call(x=None) == tla.EINVAL and call(r=None) == tla.EINVAL
    for who in ("x", "f", "gate", "scale", "post_w", "pre_b", "r", "y"):
        assert call(**{who: ctypes.c_void_p(0x10000004)}) == tla.EINVAL
    assert call(r=P[1]) == tla.EINVAL and call(y=P[0]) == tla.EINVAL and call(y=P[8]) == tla.EINVAL
    assert call(r=ctypes.c_void_p(0x10000000 + 128)) == tla.EINVAL  # in place, but a row late
    assert call(r=P[0], y=P[0]) == tla.EINVAL
    assert "overlap" in lib.vggt3_last_error().decode()


def test_grad_refusals(lib):
    nb = lib.vggt3_block_join_grad_workspace_bytes(10, 64, tla.BF16)
    assert nb > 0 and lib.vggt3_block_join_grad_workspace_bytes(0, 64, tla.BF16) == 0
    assert lib.vggt3_block_join_grad_workspace_bytes(10, 8193, tla.BF16) == 0

    def call(**kw):
        a = dict(r=P[0], f=P[1], gate=P[2], per=1, scale=P[3], post=1, post_w=P[4], post_b=P[5], pre=2, pre_w=P[6], eps=1e-6,
                 dr=P[7], dy=P[8], dx=P[9], df=P[10], dgate=P[11], dscale=P[12], dpost_w=P[13], dpost_b=P[14],
                 dpre_w=P[15], dpre_b=P[16], n=10, C=64, dt=tla.F32, ws=P[17], nb=1 << 24)
        a.update(kw)
        return lib.vggt3_block_join_grad(a["r"], a["f"], a["gate"], a["per"], a["scale"], a["post"], a["post_w"], a["post_b"],
                                         a["pre"], a["pre_w"], a["eps"], a["dr"], a["dy"], a["dx"], a["df"], a["dgate"],
                                         a["dscale"], a["dpost_w"], a["dpost_b"], a["dpre_w"], a["dpre_b"], a["n"], a["C"],
                                         a["dt"], a["ws"], a["nb"], None)

    assert call(n=-1) == tla.EINVAL and call(C=9000) == tla.EUNSUPPORTED and call(dt=3) == tla.EINVAL
    assert call(ws=None) == tla.EWORKSPACE and call(nb=16) == tla.EWORKSPACE
    assert call(r=None) == tla.EINVAL and call(dy=None) == tla.EINVAL
    assert call(gate=None) == tla.EINVAL  # dgate without a gate
    assert call(f=None) == tla.EINVAL
    assert call(pre=0, pre_w=None) == tla.EINVAL  # dy without a norm
    assert call(pre=0, pre_w=None, dy=None, dpre_w=None, dpre_b=None, dr=None) == tla.EINVAL
    assert call(post=0, post_w=None, post_b=None) == tla.EINVAL  # dpost_w without a norm
    assert call(dx=P[0]) == tla.EINVAL and call(df=P[7]) == tla.EINVAL and call(dx=P[8]) == tla.EINVAL
    assert call(dscale=P[13]) == tla.EINVAL and call(ws=P[9]) == tla.EINVAL and call(dx=P[7], f=P[7]) == tla.EINVAL
    assert call(dy=ctypes.c_void_p(0x10000008)) == tla.EINVAL


def test_binding_refusals():
    x, f = torch.zeros(6, 32), torch.zeros(6, 32)
    w = torch.ones(32)
    with pytest.raises(ValueError, match="GPU"):
        tla.block_join(x, f, pre="rms")
    with pytest.raises(KeyError):
        tla.block_join(x, f, pre="batch")
    with pytest.raises(ValueError, match="match"):
        tla.block_join(x, f[:5])
    with pytest.raises(ValueError, match="match"):
        tla.block_join(x, f.bfloat16())
    with pytest.raises(ValueError, match="gate"):
        tla.block_join(x, f, gate=torch.zeros(6, 32), gate_tokens=2)
    with pytest.raises(ValueError, match="gate"):
        tla.block_join(x, f, gate=torch.zeros(6, 32, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="gate_tokens"):
        tla.block_join(x, f, gate=torch.zeros(6, 32), gate_tokens=0)
    with pytest.raises(ValueError, match="float32"):
        tla.block_join(x, f, scale=w.bfloat16())
    with pytest.raises(ValueError, match="elements"):
        tla.block_join(x, f, post="rms", post_w=w[:31])
    with pytest.raises(ValueError, match="norm"):
        tla.block_join(x, f, mx4=True)
    with pytest.raises(ValueError, match="block output"):
        tla.block_join(x, pre="rms", r=f)
    with pytest.raises(ValueError, match="GPU"):
        tla.block_join_grad(x, f, dr=f, scale=w)
    with pytest.raises(ValueError, match="match"):
        tla.block_join_grad(x, f, dr=f[:3])
    with pytest.raises(ValueError, match="dgate"):
        tla.block_join_grad(x, f, dr=f, out=tla.BlockJoinGrads(dgate=x))


@pytest.mark.parametrize("per", [2 ** 31, 2 ** 63 - 1, 2 ** 63, 2 ** 64 + 1, 2 ** 64 + 2])
def test_gate_group_longer_than_any_run_of_tokens(per, monkeypatch):
    # one gate row serves all tokens; the count that the C call sees must not wrap to a small one, which would have it
    # read gate rows that are not there
    seen = []
    monkeypatch.setattr(tla, "_pointers", lambda *ts: (0, [None if t is None else 0x10000 for t in ts]))
    monkeypatch.setattr(tla, "_run", lambda name, dev, *args: seen.append(args[3]))
    x, gate = torch.zeros(6, 32), torch.zeros(1, 32)
    tla.block_join(x, x.clone(), gate, per)
    tla.block_join_grad(x, x.clone(), x.clone(), gate=gate, gate_tokens=per)
    assert len(seen) == 2
    for v in seen:
        assert ctypes.c_int64(v).value >= 6


def test_y_of_the_other_form_is_refused():
    x = torch.zeros(4, 64)
    y4 = tla.Mx4(torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(1, 1, 64, 4, dtype=torch.uint8), 64)
    with pytest.raises(TypeError, match="mx4"):
        tla.block_join(x, x.clone(), pre="rms", y=y4)
    with pytest.raises(TypeError, match="Mx4"):
        tla.block_join(x, x.clone(), pre="rms", y=x.clone(), mx4=True)


@pytest.mark.parametrize("where", ["post", "pre"])
def test_unknown_norm_says_which_there_are(where):
    x = torch.zeros(4, 64)
    with pytest.raises(KeyError, match="batch.*rms.*layer"):
        tla.block_join(x, x.clone(), **{where: "batch"})
    with pytest.raises(KeyError, match="batch.*rms.*layer"):
        tla.block_join_grad(x, x.clone(), x.clone(), **{where: "batch"})
