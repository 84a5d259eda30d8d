"""The gated delta rule over sequences whose rows lie in any order, on the GPU.

A sequence that ends before it begins is empty, wherever it stands in the list. Tolerances are those of test_gpu_delta.py.
"""
import numpy as np
import pytest
import torch

import test_layer_amd as tla
from test_gpu_delta import _case, _check_forward, _check_grad

pytestmark = pytest.mark.gpu
CODE = {"bf16": tla.BF16, "f32": tla.F32}


def _ordered(cu, n, hk, group, dk, dv, dtype, seed):
    """A case of n rows with these boundaries (and as many states as sequences)."""
    nseq = len(cu) - 1
    c = _case([n] + [0] * (nseq - 1), hk, group, dk, dv, dtype, seed=seed)
    return dict(c, cu=torch.tensor(cu, dtype=torch.int32).cuda())


def _unwritten(grad, c, dtype):
    """A workspace of NaN: what is read there before it was written shows."""
    hv, dk, dv = c["dims"]
    size = tla.gated_delta_grad_workspace_bytes if grad else tla.gated_delta_workspace_bytes
    return torch.full((size(c["n"], len(c["lens"]), 0, c["heads"], hv, dk, dv, CODE[dtype]),), 0xFF, dtype=torch.uint8, device="cuda")


def _check(cu, n, hk, group, dk, dv, seed=0):
    c = _ordered(cu, n, hk, group, dk, dv, "f32", seed)
    _check_forward(c, workspace=_unwritten(False, c, "f32"))
    _check_grad(c, workspace=_unwritten(True, c, "f32"))


@pytest.mark.parametrize("cu,n", [([90, 10, 100], 100), ([100, 200, 0, 100], 200), ([60, 100, 0, 60], 100), ([64, 32, 100], 110),
                                  ([600, 900, 300, 600, 0, 300], 905)], ids=str)
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
def test_boundaries_that_decrease(cu, n, dk, dv):
    _check(cu, n, 1, 2, dk, dv)


def _backwards(lens):
    ends = np.concatenate([[0], np.cumsum(lens)])
    return [int(x) for i in reversed(range(len(lens))) for x in (ends[i], ends[i + 1])]


@pytest.mark.parametrize("blocks", [5, 32, 33, 128, 129, 200])
def test_blocks_of_rows_backwards(blocks):
    # 9, 63, 65, 255, 257 and 399 sequences, every other one empty
    lens = np.random.default_rng(blocks).integers(0, 70, blocks)
    _check(_backwards(lens), int(lens.sum()) + 3, 1, 2, 64, 64, seed=blocks)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[40, 0, 33, 64], [300, 500, 299], [9] * 100, [7] * 2100], ids=["short", "cut", "some", "many"])
def test_the_same_sequences_in_both_orders(lens, dtype):
    # bit for bit: the order of the list decides nothing but the order of the states
    down = _backwards(lens)
    n, blocks = sum(lens), len(lens)
    ends = np.concatenate([[0], np.cumsum(lens)])
    up = [int(x) for e in ends for x in (e, e)][1:-1]  # every other one empty here too
    c = _ordered(up, n, 2, 2, 64, 64, dtype, 1)
    turn = torch.arange(2 * blocks - 2, -1, -1)
    r = dict(c, cu=torch.tensor(down, dtype=torch.int32).cuda(), state=c["state"][turn].contiguous(), dstate=c["dstate"][turn].contiguous())

    def run(x):
        args = (x["q"], x["k"], x["v"], x["g"], x["beta"])
        o, s = tla.gated_delta(*args, 2, state=x["state"], cu_seqlens=x["cu"], workspace=_unwritten(False, x, dtype))
        g = tla.gated_delta_grad(*args, x["do"], 2, dstate=x["dstate"], state=x["state"], cu_seqlens=x["cu"],
                                 workspace=_unwritten(True, x, dtype))
        return (o, *g[:5]), (s, g.dstate)

    for a, b in zip(run(c), run(r)):
        for x, y in zip(a, b):
            assert torch.isfinite(x).all()
            assert torch.equal(x, y if x.dim() == 2 else y[turn])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_shared_heads_in_many_sequences(dtype):
    # a shared key head's gradients in more sequences than a workgroup has threads, and rows of no sequence behind them
    lens = np.random.default_rng(9).integers(0, 4, 3000).tolist()
    lens[1234], lens[2999] = 100, 33
    c = _case(lens, 1, 2, 64, 64, dtype, state=False, seed=9, behind=40)
    out = tla.GatedDeltaGrads(*(torch.full_like(c[x], 5.0) for x in ("q", "k", "v", "g", "beta")))
    got = _check_grad(c, out=out)
    for x in got[:5]:
        assert (x[c["n"]:] == 5.0).all()


@pytest.mark.parametrize("nseq", [40, 100, 300])
def test_boundaries_that_change_between_replays(nseq):
    # a captured call whose boundaries' tensor gets other values, in order and not: numbers are counted anew each time
    n = 900
    c = _ordered([0] * nseq + [n], n, 1, 2, 64, 64, "f32", 4)
    r = np.random.default_rng(nseq)

    def order(turn):
        ends = np.sort(r.integers(0, n + 1, nseq // 2 + 1))
        cu = np.concatenate([[x, y] for x, y in zip(ends, ends[1:])][::-1 if turn % 2 else 1])
        return torch.tensor(np.concatenate([cu, np.repeat(cu[-1], nseq + 1 - len(cu))]), dtype=torch.int32)

    def run():
        args = (c["q"], c["k"], c["v"], c["g"], c["beta"])
        kw = dict(state=c["state"], cu_seqlens=c["cu"])
        o = torch.zeros_like(c["v"])
        out = tla.GatedDeltaGrads(*(torch.zeros_like(c[x]) for x in ("q", "k", "v", "g", "beta")), torch.empty_like(c["state"]))
        o, s = tla.gated_delta(*args, 1, out=o, **kw)
        return o, s, *tla.gated_delta_grad(*args, c["do"], 1, dstate=c["dstate"], out=out, **kw)

    c["cu"].copy_(order(0))
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = run()
    for turn in range(5):
        c["cu"].copy_(order(turn))
        g.replay()
        torch.cuda.synchronize()
        for x, y in zip(got, run()):
            assert torch.isfinite(x).all() and torch.equal(x, y), turn
