"""Refusals of the gated delta rule and of the query/key preparation, on the host."""
import ctypes

import pytest
import torch

import test_layer_amd as tla
from test_layer_amd import _lib

P = [ctypes.c_void_p(0x10000000 * (i + 1)) for i in range(32)]


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def _delta(lib, **kw):
    a = dict(q=P[0], k=P[1], v=P[2], g=P[3], beta=P[4], cu=P[5], longest=0, state=P[6], scale=1.0, o=P[7], so=P[8], n=100, nseq=3,
             hk=2, hv=4, dk=64, dv=64, dt=tla.BF16, ws=P[9], nb=1 << 27)
    a.update(kw)
    return lib.vggt3_gated_delta(a["q"], a["k"], a["v"], a["g"], a["beta"], a["cu"], a["longest"], a["state"], a["scale"], a["o"],
                                 a["so"], a["n"], a["nseq"], a["hk"], a["hv"], a["dk"], a["dv"], a["dt"], a["ws"], a["nb"], None)


SHAPES = [(dict(dt=2), tla.EINVAL), (dict(n=-1), tla.EINVAL), (dict(n=1 << 31), tla.EUNSUPPORTED), (dict(hk=0), tla.EINVAL),
          (dict(hv=3), tla.EINVAL), (dict(hv=0), tla.EINVAL), (dict(dk=32), tla.EUNSUPPORTED), (dict(dv=96), tla.EUNSUPPORTED),
          (dict(dk=0), tla.EUNSUPPORTED), (dict(hk=1, hv=1025), tla.EUNSUPPORTED), (dict(scale=float("nan")), tla.EINVAL),
          (dict(scale=float("inf")), tla.EINVAL), (dict(beta=None), tla.EINVAL), (dict(q=None), tla.EINVAL),
          (dict(k=None), tla.EINVAL), (dict(v=None), tla.EINVAL)]
SEQS = [(dict(nseq=0), tla.EINVAL), (dict(cu=None), tla.EINVAL), (dict(longest=-1), tla.EINVAL),
        (dict(nseq=1 << 23, nb=1 << 62), tla.EUNSUPPORTED)]


def test_delta_refusals(lib):
    for kw, rc in SHAPES + SEQS + [(dict(o=None), tla.EINVAL)]:
        assert _delta(lib, **kw) == rc, kw
    for who in ("q", "k", "v", "state", "o", "so"):
        assert _delta(lib, **{who: ctypes.c_void_p(0x10000004)}) == tla.EINVAL, who
    for who in ("g", "beta", "cu"):
        assert _delta(lib, **{who: ctypes.c_void_p(0x10000002)}) == tla.EINVAL, who
    assert _delta(lib, o=P[2]) == tla.EINVAL and _delta(lib, so=P[7]) == tla.EINVAL and _delta(lib, o=P[6]) == tla.EINVAL
    assert _delta(lib, so=ctypes.c_void_p(P[6].value + 16384)) == tla.EINVAL  # in place, but a head late
    need = lib.vggt3_gated_delta_workspace_bytes(1000, 1, 0, 2, 4, 64, 64, tla.BF16)
    # a sequence that may be long is cut, and its pieces' states lie there
    assert need > lib.vggt3_gated_delta_workspace_bytes(1000, 1, 64, 2, 4, 64, 64, tla.BF16) > 0
    assert _delta(lib, n=1000, nseq=1, nb=need - 1) == tla.EWORKSPACE and _delta(lib, n=1000, nseq=1, ws=None) == tla.EWORKSPACE
    assert _delta(lib, n=1000, nseq=1, ws=P[7]) == tla.EINVAL
    assert lib.vggt3_gated_delta_workspace_bytes(1000, 1, 0, 2, 4, 63, 64, tla.BF16) == 0


def _delta_grad(lib, **kw):
    a = dict(q=P[0], k=P[1], v=P[2], g=P[3], beta=P[4], cu=P[5], longest=0, state=P[6], scale=1.0, do=P[7], dso=P[8], dq=P[9],
             dko=P[10], dvo=P[11], dg=P[12], db=P[13], ds=P[14], n=100, nseq=3, hk=2, hv=4, dk=64, dv=64, dt=tla.F32, ws=P[15],
             nb=1 << 27)
    a.update(kw)
    return lib.vggt3_gated_delta_grad(a["q"], a["k"], a["v"], a["g"], a["beta"], a["cu"], a["longest"], a["state"], a["scale"],
                                      a["do"], a["dso"], a["dq"], a["dko"], a["dvo"], a["dg"], a["db"], a["ds"], a["n"], a["nseq"],
                                      a["hk"], a["hv"], a["dk"], a["dv"], a["dt"], a["ws"], a["nb"], None)


def test_delta_grad_refusals(lib):
    for kw, rc in SHAPES + SEQS + [(dict(do=None), tla.EINVAL), (dict(g=None), tla.EINVAL)]:
        assert _delta_grad(lib, **kw) == rc, kw
    for who in ("q", "k", "v", "state", "do", "dso", "dq", "dko", "dvo", "ds", "ws"):
        assert _delta_grad(lib, **{who: ctypes.c_void_p(0x10000004)}) == tla.EINVAL, who
    assert _delta_grad(lib, dq=P[0]) == tla.EINVAL and _delta_grad(lib, dg=P[13]) == tla.EINVAL
    assert _delta_grad(lib, dvo=P[7]) == tla.EINVAL and _delta_grad(lib, ds=P[6]) == tla.EINVAL
    assert _delta_grad(lib, ws=P[9]) == tla.EINVAL
    need = lib.vggt3_gated_delta_grad_workspace_bytes(100, 3, 0, 2, 4, 64, 64, tla.F32)
    assert _delta_grad(lib, nb=need - 1) == tla.EWORKSPACE and _delta_grad(lib, ws=None) == tla.EWORKSPACE


def _step(lib, **kw):
    a = dict(q=P[0], k=P[1], v=P[2], g=P[3], beta=P[4], state=P[5], slots_n=20, slots=P[6], scale=1.0, o=P[7], n=10, hk=2, hv=4,
             dk=64, dv=128, dt=tla.BF16)
    a.update(kw)
    return lib.vggt3_gated_delta_step(a["q"], a["k"], a["v"], a["g"], a["beta"], a["state"], a["slots_n"], a["slots"], a["scale"],
                                      a["o"], a["n"], a["hk"], a["hv"], a["dk"], a["dv"], a["dt"], None)


def test_step_refusals(lib):
    for kw, rc in SHAPES + [(dict(o=None), tla.EINVAL), (dict(state=None), tla.EINVAL), (dict(slots_n=-1), tla.EINVAL),
                            (dict(slots=None, slots_n=9), tla.EINVAL), (dict(n=1 << 22), tla.EUNSUPPORTED)]:
        assert _step(lib, **kw) == rc, kw
    assert _step(lib, n=0) == tla.OK
    assert _step(lib, o=P[5]) == tla.EINVAL and _step(lib, state=P[2]) == tla.EINVAL
    for who in ("q", "k", "v", "state", "o"):
        assert _step(lib, **{who: ctypes.c_void_p(0x10000008)}) == tla.EINVAL, who
    assert _step(lib, slots=ctypes.c_void_p(0x10000002)) == tla.EINVAL


def _sections(*s):
    return (ctypes.c_int32 * len(s))(*s) if s else None


def _qk(lib, **kw):
    a = dict(q=P[0], qs=256, k=P[1], ks=128, norm=1, qw=P[2], qb=P[3], kw=P[4], kb=P[5], eps=1e-6, pos=P[6], sec=(16, 16),
             base=100.0, per=1, inter=0, qo=P[7], ko=P[8], n=10, h=4, hk=2, d=64, dt=tla.BF16)
    a.update(kw)
    axes = a.get("axes", len(a["sec"]))
    return lib.vggt3_qk_norm_rope(a["q"], a["qs"], a["k"], a["ks"], a["norm"], a["qw"], a["qb"], a["kw"], a["kb"], a["eps"],
                                  a["pos"], _sections(*a["sec"]), axes, a["base"], a["per"], a["inter"], a["qo"], a["ko"], a["n"],
                                  a["h"], a["hk"], a["d"], a["dt"], None)


QK = [(dict(dt=2), tla.EINVAL), (dict(n=-1), tla.EINVAL), (dict(n=(1 << 31) + 1), tla.EUNSUPPORTED), (dict(h=0), tla.EINVAL),
      (dict(hk=-1), tla.EINVAL), (dict(d=0), tla.EINVAL), (dict(d=513), tla.EUNSUPPORTED), (dict(norm=4), tla.EINVAL),
      (dict(norm=-1), tla.EINVAL), (dict(eps=-1.0), tla.EINVAL), (dict(eps=float("nan")), tla.EINVAL),
      (dict(sec=(16, 17)), tla.EINVAL), (dict(sec=(0, 16)), tla.EINVAL), (dict(sec=(1,) * 5), tla.EUNSUPPORTED),
      (dict(sec=(), axes=1), tla.EINVAL), (dict(axes=-1), tla.EINVAL), (dict(sec=(2 ** 31 - 1, 2 ** 31 - 1)), tla.EINVAL),
      (dict(base=0.0), tla.EINVAL), (dict(base=-1.0), tla.EINVAL), (dict(base=float("inf")), tla.EINVAL), (dict(pos=None), tla.EINVAL),
      (dict(norm=0, qw=None, kw=None, qb=None, kb=None, sec=(), pos=None), tla.EINVAL), (dict(norm=3), tla.EINVAL),
      (dict(norm=0), tla.EINVAL), (dict(q=None), tla.EINVAL), (dict(k=None), tla.EINVAL), (dict(qs=255), tla.EINVAL),
      (dict(ks=(1 << 31) + 1), tla.EINVAL), (dict(hk=0), tla.EINVAL)]


def test_qk_refusals(lib):
    for kw, rc in QK + [(dict(qo=None), tla.EINVAL), (dict(ko=None), tla.EINVAL)]:
        assert _qk(lib, **kw) == rc, kw
    assert _qk(lib, n=0) == tla.OK
    assert _qk(lib, hk=0, k=None, kw=None, kb=None) == tla.EINVAL  # k_out without keys
    assert _qk(lib, qo=P[1]) == tla.EINVAL and _qk(lib, qo=P[8]) == tla.EINVAL and _qk(lib, ko=P[6]) == tla.EINVAL
    assert _qk(lib, qo=P[0], qs=320) == tla.EINVAL  # in place, rows with gaps
    assert _qk(lib, qo=ctypes.c_void_p(P[0].value + 128)) == tla.EINVAL
    assert _qk(lib, q=ctypes.c_void_p(0x10000001)) == tla.EINVAL and _qk(lib, qw=ctypes.c_void_p(0x10000002)) == tla.EINVAL


def test_qk_grad_refusals(lib):
    def call(**kw):
        a = dict(q=P[0], qs=256, k=P[1], ks=128, dqo=P[2], dko=P[3], norm=1, qw=P[4], kw=P[5], eps=1e-6, pos=P[6], sec=(16, 16),
                 base=100.0, per=1, inter=0, dq=P[7], dk=P[8], dqw=P[9], dqb=P[10], dkw=P[11], dkb=P[12], n=10, h=4, hk=2, d=64,
                 dt=tla.BF16, ws=P[13], nb=1 << 24)
        a.update(kw)
        axes = a.get("axes", len(a["sec"]))
        return lib.vggt3_qk_norm_rope_grad(a["q"], a["qs"], a["k"], a["ks"], a["dqo"], a["dko"], a["norm"], a["qw"], a["kw"],
                                           a["eps"], a["pos"], _sections(*a["sec"]), axes, a["base"], a["per"], a["inter"], a["dq"],
                                           a["dk"], a["dqw"], a["dqb"], a["dkw"], a["dkb"], a["n"], a["h"], a["hk"], a["d"], a["dt"],
                                           a["ws"], a["nb"], None)

    for kw, rc in [(x, r) for x, r in QK if "qb" not in x] + [(dict(dqo=None), tla.EINVAL), (dict(dko=None), tla.EINVAL)]:
        assert call(**kw) == rc, kw
    assert call(norm=3, qw=None, kw=None) == tla.EINVAL  # gradients of weights without a norm that has them
    assert call(ws=None) == tla.EWORKSPACE and call(nb=16) == tla.EWORKSPACE
    assert call(dq=P[0]) == tla.EINVAL and call(dq=P[3]) == tla.EINVAL and call(dqw=P[10]) == tla.EINVAL
    assert call(ws=P[7]) == tla.EINVAL


def test_binding_refusals():
    q, v = torch.zeros(6, 128), torch.zeros(6, 256)
    g = torch.zeros(6, 4)
    s = torch.zeros(1, 4, 64, 64)
    cu = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        tla.gated_delta(q, q.clone(), v, g, g, 2)
    for bad, what in ((dict(k=q[:5]), "match"), (dict(v=v[:5]), "match"), (dict(v=v.bfloat16()), "match"), (dict(beta=g[:5]), "beta"),
                      (dict(beta=g.bfloat16()), "beta"), (dict(g=g[:, :3]), "match"), (dict(beta=torch.zeros(6, 3), g=None), "heads"),
                      (dict(n_heads=3), "heads"), (dict(n_heads=0), "heads"), (dict(v=torch.zeros(6, 192), beta=torch.zeros(6, 3), g=None),
                                                                              "multiple"), (dict(v=torch.zeros(6, 0)), "heads")):
        a = dict(q=q, k=q.clone(), v=v, g=g, beta=g, n_heads=2)
        a.update(bad)
        with pytest.raises(ValueError, match=what):
            tla.gated_delta(**a)
        with pytest.raises(ValueError, match=what):
            tla.gated_delta_grad(**a, d_o=a["v"])
        with pytest.raises(ValueError, match=what):
            tla.gated_delta_step(**a, state=s)
    k = q.clone()
    for bad, what in ((dict(state=s[0]), "state"), (dict(state=s.double()), "state"), (dict(state=s.expand(2, 4, 64, 64)), "state"),
                      (dict(cu_seqlens=cu.long()), "cu_seqlens"), (dict(cu_seqlens=cu[:1]), "cu_seqlens"), (dict(max_seqlen=-1), "max_seqlen")):
        with pytest.raises(ValueError, match=what):
            tla.gated_delta(q, k, v, g, g, 2, **bad)
        with pytest.raises(ValueError, match=what):
            tla.gated_delta_grad(q, k, v, g, g, v, 2, **bad)
    with pytest.raises(ValueError, match="out"):
        tla.gated_delta(q, k, v, g, g, 2, out=q)
    with pytest.raises(ValueError, match="state_out"):
        tla.gated_delta(q, k, v, g, g, 2, state_out=s[0])
    with pytest.raises(ValueError, match="d_o"):
        tla.gated_delta_grad(q, k, v, g, g, v[:4], 2)
    with pytest.raises(ValueError, match="dstate"):
        tla.gated_delta_grad(q, k, v, g, g, v, 2, dstate=s[0])
    with pytest.raises(ValueError, match="dg without"):
        tla.gated_delta_grad(q, k, v, None, g, v, 2, out=tla.GatedDeltaGrads(dg=g))
    with pytest.raises(ValueError, match="dk"):
        tla.gated_delta_grad(q, k, v, g, g, v, 2, out=tla.GatedDeltaGrads(dk=v))
    with pytest.raises(ValueError, match="slots"):
        tla.gated_delta_step(q, k, v, g, g, 2, s, slots=torch.zeros(6, dtype=torch.int64))
    with pytest.raises(ValueError, match="states"):
        tla.gated_delta_step(q, k, v, g, g, 2, s)
    with pytest.raises(ValueError, match="state"):
        tla.gated_delta_step(q, k, v, g, g, 2, s[0])


def test_qk_binding_refusals():
    q, k, w = torch.zeros(6, 256), torch.zeros(6, 128), torch.ones(64)
    pos = torch.zeros(6, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        tla.qk_norm_rope(q, k, 4, 2)
    for bad, what in ((dict(n_heads=3), "heads"), (dict(n_heads_k=4), "expected"), (dict(k=k[:4]), "match"), (dict(k=k.bfloat16()), "match"),
                      (dict(pos=pos), "together"), (dict(sections=(16, 16)), "together"), (dict(pos=pos, sections=(16,)), "pos"),
                      (dict(pos=pos.long(), sections=(16, 16)), "pos"), (dict(q_w=w[:32], norm="rms"), "elements"),
                      (dict(k_w=w.bfloat16(), norm="rms"), "float32"), (dict(k=None, k_w=w, norm="rms"), "without k")):
        a = dict(q=q, k=k, n_heads=4, n_heads_k=2)
        a.update(bad)
        with pytest.raises(ValueError, match=what):
            tla.qk_norm_rope(**a)
        with pytest.raises(ValueError, match=what):
            tla.qk_norm_rope_grad(**a, dq_out=a["q"], dk_out=a["k"])
    with pytest.raises(KeyError, match="batch.*l2.*layer"):
        tla.qk_norm_rope(q, k, 4, 2, norm="batch")
    with pytest.raises(KeyError, match="batch.*l2.*layer"):
        tla.qk_norm_rope_grad(q, k, q, k, 4, 2, norm="batch")
    with pytest.raises(ValueError, match="q_out"):
        tla.qk_norm_rope(q, k, 4, 2, q_out=k)
    with pytest.raises(ValueError, match="k_out without"):
        tla.qk_norm_rope(q, None, 4, k_out=k)
    with pytest.raises(ValueError, match="together"):
        tla.qk_norm_rope_grad(q, k, q, None, 4, 2)
    with pytest.raises(ValueError, match="without k"):
        tla.qk_norm_rope_grad(q, None, q, None, 4, out=tla.QkNormRopeGrads(dk=k))
