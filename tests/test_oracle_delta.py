"""Pins of the gated delta rule's oracle: closed forms, its products of rank-one steps, every gradient against central
differences; and a model of how sequences are numbered in pieces."""
import numpy as np
import pytest

from oracle import delta


def _inputs(n=6, dk=4, dv=3, seed=0):
    g = np.random.default_rng(seed)
    q, k = g.standard_normal((2, n, dk))
    return dict(q=q, k=k, v=g.standard_normal((n, dv)), g=-np.exp(g.standard_normal(n)), beta=g.uniform(0, 1, n),
                S=g.standard_normal((dk, dv)))


def test_state_is_the_product_of_its_steps():
    p = _inputs()
    _, S = delta.forward(**p)
    M, R = np.eye(4), np.zeros((4, 3))
    for t in range(6):
        A = np.exp(p["g"][t]) * (np.eye(4) - p["beta"][t] * np.outer(p["k"][t], p["k"][t]))
        M, R = A @ M, A @ R + p["beta"][t] * np.outer(p["k"][t], p["v"][t])
    assert np.allclose(S, M @ p["S"] + R, rtol=1e-12, atol=1e-12)


def test_orthonormal_keys_store_and_return_their_values():
    k = np.eye(4)
    v = np.random.default_rng(1).standard_normal((4, 3))
    o, S = delta.forward(k, k, v, np.zeros(4), np.ones(4))
    assert np.allclose(o, v) and np.allclose(S, v)
    # a full step onto a stored key replaces its value
    o, S = delta.forward(k[:1], k[:1], 2 * v[:1], np.zeros(1), np.ones(1), S)
    assert np.allclose(S[0], 2 * v[0]) and np.allclose(S[1:], v[1:])


def test_one_step_is_gradient_descent_on_the_squared_error():
    p = _inputs(1)
    L = lambda S: 0.5 * np.sum((S.T @ p["k"][0] - p["v"][0]) ** 2)  # noqa: E731
    grad = np.zeros((4, 3))
    for i in np.ndindex(4, 3):
        e = np.zeros((4, 3))
        e[i] = 1e-6
        grad[i] = (L(p["S"] + e) - L(p["S"] - e)) / 2e-6
    _, S = delta.forward(p["q"], p["k"], p["v"], np.zeros(1), p["beta"], p["S"])
    assert np.allclose(S, p["S"] - p["beta"][0] * grad, rtol=1e-8, atol=1e-8)


def test_an_infinite_decay_forgets():
    p = _inputs()
    p["g"][3] = -np.inf
    o, S = delta.forward(**p)
    fresh = {x: (None if x == "S" else p[x][3:]) for x in p}
    fresh["g"] = np.concatenate([[0.0], p["g"][4:]])
    o2, S2 = delta.forward(**fresh)
    assert np.array_equal(o[3:], o2) and np.array_equal(S, S2)


@pytest.mark.parametrize("heads,group", [(1, 1), (2, 1), (2, 3)])
def test_gradients_against_differences(heads, group):
    g = np.random.default_rng(3)
    n, dk, dv, hv, cu = 7, 3, 2, heads * group, [0, 3, 3, 7]
    p = dict(q=g.standard_normal((n, heads * dk)), k=g.standard_normal((n, heads * dk)), v=g.standard_normal((n, hv * dv)),
             g=-np.exp(g.standard_normal((n, hv))), beta=g.uniform(0, 1, (n, hv)), S=g.standard_normal((3, hv, dk, dv)))
    do, dS = g.standard_normal((n, hv * dv)), g.standard_normal((3, hv, dk, dv))

    def loss(x):
        o, last = delta.run(x["q"], x["k"], x["v"], x["g"], x["beta"], heads, x["S"], 0.7, cu)
        return (o * do).sum() + (last * dS).sum()

    got = delta.run(p["q"], p["k"], p["v"], p["g"], p["beta"], heads, p["S"], 0.7, cu, do, dS)
    for name, x in p.items():
        num = np.zeros_like(x)
        for i in np.ndindex(x.shape):
            t = dict(p, **{name: x.copy()})
            t[name][i] += 1e-6
            hi = loss(t)
            t[name][i] -= 2e-6
            num[i] = (hi - loss(t)) / 2e-6
        # central differences at 1e-6: truncation ~1e-12, rounding ~1e-16 / 1e-6 of a loss of order 100
        assert np.allclose(got["d" + (name if name != "S" else "state")], num, rtol=1e-6, atol=1e-6), name


def _bound(cu, i, n):
    return min(max(cu[i], 0), n)


def _find(cu, n, per, sid):
    """A lane-for-lane model of the kernels' search for piece sid: (sequence, piece or -1, first row, rows)."""
    nseq = len(cu) - 1
    lo, size = 0, nseq
    if nseq < 64:  # a boundary a lane
        lo = max(sum(_bound(cu, i, n) // per + i <= sid for i in range(nseq)) - 1, 0)
        size = 1
    while size > 1:
        stride = (size + 63) // 64
        before = [lane * stride < size and _bound(cu, lo + lane * stride, n) // per + lo + lane * stride <= sid
                  for lane in range(64)]
        found = sum(before)
        lo += max(found - 1, 0) * stride
        size = min(size, stride)
        if lo + size > nseq:
            size = nseq - lo
    begin, end = _bound(cu, lo, n), _bound(cu, lo + 1, n)
    length = max(end - begin, 0)
    seg = sid - (begin // per + lo)
    segs = -(-length // per) if length > 0 else 1
    left = length - seg * per
    if seg < 0 or seg >= segs:
        return lo, -1, 0, 0
    return lo, seg, begin + seg * per, max(0, min(left, per))


@pytest.mark.parametrize("seed", range(12))
def test_pieces_cover_every_row_once(seed):
    g = np.random.default_rng(seed)
    nseq = [1, 2, 3, 63, 64, 65, 200, 4096, 4100, 5000, 7, 30][seed]
    lens = g.integers(0, 90, nseq) * (g.random(nseq) < 0.7)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(int)
    n = int(cu[-1]) + int(g.integers(0, 70))  # rows of no sequence behind the last
    for per in (32, 96, (n // 32 + 1) * 32):
        rows, seen = np.zeros(n, int), set()
        for sid in range(n // per + nseq):
            b, seg, first, length = _find(cu, n, per, sid)
            if seg < 0:
                continue
            assert (b, seg) not in seen and cu[b] <= first and first + length <= cu[b + 1]
            seen.add((b, seg))
            rows[first:first + length] += 1
        assert (rows[:cu[-1]] == 1).all() and (rows[cu[-1]:] == 0).all()
        assert {b for b, seg in seen if seg == 0} == set(range(nseq))  # empty sequences too


@pytest.mark.parametrize("cu", [[0, 40, 1000], [-5, 20, 50], [0, 60, 30, 70], [90, 10, 100], [7, 7, 7], [2 ** 31 - 1, 0, -3]])
def test_bad_boundaries_stay_inside(cu):
    n = 77
    for per in (32, 96):
        for sid in range(n // per + len(cu) - 1):
            b, seg, first, length = _find(cu, n, per, sid)
            if seg >= 0:
                assert 0 <= first and first + length <= n
                # the chunk's place in a buffer of n / 32 + sequences
                base = _bound(cu, b, n)
                assert 0 <= base // 32 + b + (first - base) // 32 + max(0, -(-length // 32) - 1) < n // 32 + len(cu) - 1
