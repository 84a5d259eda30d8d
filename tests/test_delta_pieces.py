"""How the gated delta rule's kernels number pieces and chunks: a lane-for-lane model on the host, for sequences in any order."""
import numpy as np
import pytest

CHUNK = 32


def _bound(cu, i, n):
    return min(max(int(cu[i]), 0), n)


def _count(begin, end, per):
    return (end - begin - 1) // per + 1 if end > begin else 1


def _firsts(cu, n, per, room):
    """The numbers of the sequences' first pieces: by their rows where boundaries are in order, counted otherwise, and of
    many sequences counted beforehand up to the room there is."""
    nseq = len(cu) - 1
    at = [_bound(cu, b, n) for b in range(nseq + 1)]
    if nseq < 256 and all(x <= y for x, y in zip(at, at[1:])):
        return np.array([x // per + b for b, x in enumerate(at[:-1])])
    first = np.concatenate([[0], np.cumsum([_count(x, y, per) for x, y in zip(at, at[1:])])])[:-1]
    return first if nseq < 256 else np.minimum(first, room)


def _find(cu, n, per, sid, pieces):
    """(sequence, piece or -1, first row, rows, number of the first chunk) of piece `sid`."""
    nseq = len(cu) - 1
    room = n // CHUNK + nseq
    first, chunk = _firsts(cu, n, per, pieces), _firsts(cu, n, CHUNK, room)
    lo, size = 0, nseq
    if nseq < 256:
        lo, size = max(sum(first <= sid) - 1, 0), 1
    while size > 1:
        stride = (size + 63) // 64
        found = sum(lane * stride < size and first[lo + lane * stride] <= sid for lane in range(64))
        lo += max(found - 1, 0) * stride
        size = min(size, stride)
        if lo + size > nseq:
            size = nseq - lo
    begin, end = _bound(cu, lo, n), _bound(cu, lo + 1, n)
    seg = sid - int(first[lo])
    slot = int(chunk[lo]) + seg * per // CHUNK
    if seg < 0 or seg >= _count(begin, end, per) or slot >= room:
        return lo, -1, begin, 0, slot
    left = max(end - begin, 0) - seg * per
    return lo, seg, begin + seg * per, min(left, per, (room - slot) * CHUNK), slot


def _walk(cu, n, per):
    pieces = n // per + len(cu) - 1
    return [x for sid in range(pieces) if (x := _find(cu, n, per, sid, pieces))[1] >= 0]


ORDERS = [[90, 10, 100], [100, 200, 0, 100], [60, 100, 0, 60], [64, 32, 100], [-5, 20, 1000, 20], [150, 200, 100, 150, 0, 100], [7, 7, 7]]


def _check(cu, n):
    nseq = len(cu) - 1
    rows = np.zeros(n, int)
    for b in range(nseq):
        rows[_bound(cu, b, n):max(_bound(cu, b + 1, n), _bound(cu, b, n))] += 1
    assert rows.max(initial=0) <= 1  # sequences share no rows
    # every chunk has matrices of its own
    chunks = {}
    for b, seg, first, length, slot in _walk(cu, n, CHUNK):
        assert slot not in chunks
        chunks[slot] = (b, first, length)
    for per in (CHUNK, 96, (n // CHUNK + 1) * CHUNK):
        seen, got = set(), np.zeros(n, int)
        for b, seg, first, length, slot in _walk(cu, n, per):
            assert (b, seg) not in seen and 0 <= first and first + length <= n
            seen.add((b, seg))
            got[first:first + length] += 1
            for i in range(0, length, CHUNK):  # and its pieces read these
                assert chunks[slot + i // CHUNK] == (b, first + i, min(CHUNK, length - i))
        assert (got == rows).all()
        assert {b for b, seg in seen if seg == 0} == set(range(nseq))  # empty sequences have their states


@pytest.mark.parametrize("cu", ORDERS, ids=str)
def test_boundaries_in_any_order(cu):
    _check(cu, 200)


@pytest.mark.parametrize("nseq", [1, 2, 31, 63, 64, 65, 129, 255, 256, 257, 700])
def test_sequences_in_any_order(nseq):
    g = np.random.default_rng(nseq)
    ends = np.concatenate([[0], np.cumsum(g.integers(0, 90, (nseq + 1) // 2))])
    # blocks of rows backwards, so that what lies between two of them in the list ends before it begins
    cu = np.concatenate([[ends[i], ends[i + 1]] for i in reversed(range(len(ends) - 1))])[:nseq + 1]
    if len(cu) < nseq + 1:
        cu = np.append(cu, 0)
    _check([int(x) for x in cu], int(ends[-1]) + 5)
    _check(sorted(int(x) for x in cu), int(ends[-1]) + 5)


@pytest.mark.parametrize("seed", range(20))
def test_boundaries_that_share_rows_stay_inside(seed):
    g = np.random.default_rng(seed)
    n, nseq = int(g.integers(1, 400)), int(g.choice([2, 5, 63, 64, 100, 300]))
    cu = g.integers(-50, n + 50, nseq + 1)
    room = n // CHUNK + nseq
    for per in (CHUNK, 96, (n // CHUNK + 1) * CHUNK):
        for b, seg, first, length, slot in _walk(cu, n, per):
            assert 0 <= first and first + length <= n and length >= 0
            assert 0 <= slot and slot + max(0, -(-length // CHUNK) - 1) < room
