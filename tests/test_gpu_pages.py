"""kv_fork, kv_compact and kv_copy against the plain loops of pages_ref.py, bit
for bit, over random histories of a table."""
import random

import numpy as np
import pytest

from . import pages_ref as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

NAMES = ("block_table", "length", "held", "refs")


def _sv():
    import greedy_speculative_decode_gb300 as sv
    return sv


def dev(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


def state(pages):
    return [getattr(pages, n).cpu().numpy().astype(np.int64) for n in NAMES]


def load(pages, arrays):
    for n, a in zip(NAMES, arrays):
        getattr(pages, n).copy_(torch.from_numpy(np.ascontiguousarray(a)).int())


def step(pages, *, out=None, source=None, keep=None, room=None):
    """One kv_fork, checked; returns its moves (None: nothing changed)."""
    sv = _sv()
    before = state(pages)
    moves = torch.full((pages.n_seq, 2), 99, dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    other = None if out is None else state(out)
    sv.kv_fork(pages, moves, source=dev(source), keep=dev(keep), room=dev(room), out=out, status=st)
    want = ref.fork(*before, source, keep, room)
    got = state(pages if out is None else out)
    if want is None:
        assert int(st.item()) & 18 and (moves.cpu().numpy() == -1).all()
        assert all(np.array_equal(a, b) for a, b in zip(got, before if out is None else other))
        return None
    assert int(st.item()) == 0
    for name, a, b in zip(NAMES, got, want):
        assert np.array_equal(a, b), (name, np.argwhere(a != b)[:5], a[a != b][:5], b[a != b][:5])
    assert np.array_equal(moves.cpu().numpy(), want[4])
    if out is not None:
        assert all(np.array_equal(a, b) for a, b in zip(state(pages), before))
    return want[4]


@pytest.mark.parametrize("n_seq,width,n_pages", [(1, 1, 1), (3, 4, 9), (8, 12, 70), (33, 7, 150), (64, 40, 1000), (300, 9, 2500),
                                                 (1024, 3, 1500)])
@pytest.mark.parametrize("in_place", [True, False])
def test_a_history_of_forks(n_seq, width, n_pages, in_place):
    sv = _sv()
    rng = random.Random(n_seq * 7 + in_place)
    pages, spare = (sv.KvPages.empty(n_seq, width, n_pages) for _ in range(2))
    failed = 0
    for k in range(30):
        length = pages.length.cpu().tolist()
        kind = rng.randrange(6)
        source = keep = room = None
        if kind in (0, 1, 5):  # go on by a few positions
            room = [min(width * 16, n + rng.choice([0, 1, 1, 5, 40])) for n in length]
        if kind == 1:  # give some back
            source = [s if rng.random() < 0.7 else -1 for s in range(n_seq)]
            room = [r if a >= 0 else 0 for r, a in zip(room, source)]
        if kind in (2, 5):  # beams
            source = [rng.randrange(n_seq) if rng.random() < 0.8 else s for s in range(n_seq)]
            room = [min(width * 16, length[a] + rng.choice([0, 3])) for a in source]
        if kind == 3:  # back to earlier positions
            keep = [rng.randrange(n + 1) if rng.random() < 0.5 else n + 7 for n in length]
        if kind == 4:  # one prompt for all
            a = rng.randrange(n_seq)
            source, keep = [a] * n_seq, [rng.choice([length[a], length[a], length[a] // 2]) for _ in range(n_seq)]
        if rng.random() < 0.5:
            source = dev(source).cpu().tolist() if source is not None else None
        got = step(pages, out=None if in_place else spare, source=source, keep=keep, room=room)
        failed += got is None
        if got is None:
            load(pages, state(pages))
            # make room: every other row goes
            step(pages, source=[s if s % 2 else -1 for s in range(n_seq)])
            continue
        if not in_place:
            pages, spare = spare, pages
        # the rows' new positions are written
        if room is not None:
            grown = [min(h * 16, max(n, r)) for n, h, r in zip(pages.length.cpu().tolist(), pages.held.cpu().tolist(), room)]
            pages.length.copy_(dev(grown))
        refs = np.zeros(n_pages, np.int64)
        t, _, h, r = state(pages)
        for s in range(n_seq):
            np.add.at(refs, t[s, :h[s]], 1)
        assert np.array_equal(refs, r)


def test_no_two_rows_write_one_page():
    """After any fork each row can go on in its last page: it is no other row's."""
    sv = _sv()
    pages = sv.KvPages.empty(6, 8, 60)
    step(pages, room=[50, 0, 0, 0, 0, 0])
    pages.length[0] = 50
    step(pages, source=[0] * 6)  # the lowest goes on in the page, five copies
    assert (pages.block_table[:, 3].unique().numel(), pages.block_table[:, 2].unique().numel()) == (6, 1)
    step(pages, source=[3, 3, 3, 4, 4, -1], keep=[50, 40, 48, 50, 33, 0])  # (a page that is full for one, begun for another)
    last = [(int(pages.length[s]) - 1) // 16 for s in range(5)]
    begun = [int(pages.block_table[s, j]) for s, j in enumerate(last) if int(pages.length[s]) % 16]
    assert all(int(pages.refs[p]) == 1 for p in begun) and len(set(begun)) == len(begun)


def test_holds_of_the_program():
    sv = _sv()
    pages = sv.KvPages.empty(2, 4, 12)
    step(pages, room=[40, 0])
    pages.length[0] = 40
    pages.refs[2] += 1  # a prefix store holds the last page too
    moves = step(pages, source=[0, -1], room=[41, 0])
    assert moves[0].tolist() == [2, 3]
    step(pages, source=[-1, -1])
    assert pages.refs.cpu().tolist() == [0, 0, 1] + [0] * 9


def test_too_few_pages_and_impossible_rows_change_nothing():
    sv = _sv()
    pages = sv.KvPages.empty(3, 4, 6)
    step(pages, room=[60, 20, 0])
    assert step(pages, room=[60, 20, 1]) is None
    assert step(pages, source=[0, 3, 2]) is None
    assert step(pages, source=[0, -2, 2]) is None
    assert step(pages, room=[65, 0, 0]) is None
    out = sv.KvPages.empty(3, 4, 6)
    assert step(pages, out=out, room=[60, 20, 1]) is None
    step(pages, source=[0, -1, 2], room=[60, 0, 1])  # pages given back are there at once


def _random_table(rng, sv, n_seq, width, n_pages):
    pages = sv.KvPages.empty(n_seq, width, n_pages)
    order = list(range(n_pages))
    rng.shuffle(order)
    table, refs = np.full((n_seq, width), -1), np.zeros(n_pages, np.int64)
    held = np.zeros(n_seq, np.int64)
    for s in range(n_seq):
        held[s] = rng.randrange(width + 1)
        for j in range(held[s]):
            p = order.pop() if order and rng.random() < 0.8 else table[s - 1, j] if s and j < held[s - 1] else -1
            if p < 0:
                held[s] = j
                break
            table[s, j] = p
            refs[p] += 1
    length = held * 16 - np.array([rng.randrange(16) if h else 0 for h in held])
    load(pages, (table, length, held, refs))
    return pages


@pytest.mark.parametrize("n_seq,width,n_pages", [(1, 1, 1), (4, 5, 33), (7, 30, 200), (60, 64, 5000), (200, 100, 70001)])
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("most", [None, 3])
def test_compact(n_seq, width, n_pages, in_place, most):
    sv = _sv()
    for seed in range(4):
        pages = _random_table(random.Random(seed), sv, n_seq, width, n_pages)
        if seed == 3:
            pages.refs[n_pages - 1] += 1  # held by the program alone
        cap = most or max(1, n_pages // 2)
        before = state(pages)
        want = ref.compact(*before, cap)
        moves = torch.full((cap, 2), 99, dtype=torch.int32, device="cuda")
        where = torch.full((n_pages,), 99, dtype=torch.int32, device="cuda") if seed % 2 else None
        out = None if in_place else sv.KvPages.empty(n_seq, width, n_pages)
        sv.kv_compact(pages, moves, where=where, out=out)
        got = state(pages if in_place else out)
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[3], want[1])
        assert np.array_equal(got[1], before[1]) and np.array_equal(got[2], before[2])
        assert np.array_equal(moves.cpu().numpy(), want[2])
        if where is not None:
            assert np.array_equal(where.cpu().numpy(), want[3])
        if most is None:
            used = int((got[3] > 0).sum())
            assert (got[3][:used] > 0).all()


POOLS = [("bf16", 1, 2, 64), ("e4m3", 1, 8, 128), ("e4m3", 16, 1, 256), ("e4m3", 16, 3, 64), ("bf16", 1, 1, 128)]


def _pool(sv, fmt, block, heads, d, n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = sv.PagedKv.empty(n, heads, d, fmt=fmt, scale_block=block)
    for t in c.tensors:
        t.view(torch.uint8).random_(0, 256, generator=g)
    return c


@pytest.mark.parametrize("fmt,block,heads,d", POOLS)
@pytest.mark.parametrize("layers", [1, 3, 40])
def test_copy(fmt, block, heads, d, layers):
    sv = _sv()
    n = 23
    caches = [_pool(sv, fmt, block, heads, d, n, k) for k in range(layers)]
    moves = dev([[1, 2], [-1, -1], [22, 0], [5, 9], [5, 10], [-1, -1]])
    want = [[t.clone() for t in c.tensors] for c in caches]
    for ts in want:
        for t in ts:
            t[[2, 0, 9, 10]] = t[[1, 22, 5, 5]]
    what = caches[0] if layers == 1 else sv.KvLayers(caches)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    sv.kv_copy(what, moves, status=st)
    assert int(st.item()) == 0
    for c, ts in zip(caches, want):
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(c.tensors, ts))
    # into other pools, of another size
    other = [_pool(sv, fmt, block, heads, d, n + 9, 100 + k) for k in range(layers)]
    want = [[t.clone() for t in c.tensors] for c in other]
    moves = dev([[4, 31], [0, 0], [4, 3]])
    for c, ts in zip(caches, want):
        for a, t in zip(c.tensors, ts):
            t[[31, 0, 3]] = a[[4, 0, 4]]
    sv.kv_copy(what, moves, into=other[0] if layers == 1 else sv.KvLayers(other), status=st)
    assert int(st.item()) == 0
    for c, ts in zip(other, want):
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(c.tensors, ts))


def test_copy_passes_over_pages_that_are_not_there():
    sv = _sv()
    c = _pool(sv, "e4m3", 1, 2, 64, 5, 0)
    want = [t.clone() for t in c.tensors]
    for t in want:
        t[3] = t[0]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    sv.kv_copy(c, dev([[0, 5], [5, 1], [-1, 2], [2, -1], [0, 3], [1 << 30, 1]]), status=st)
    assert int(st.item()) == 2
    assert all(torch.equal(a, b) for a, b in zip(c.tensors, want))


def test_a_table_with_entries_that_are_no_pages():
    sv = _sv()
    pages = sv.KvPages.empty(2, 4, 8)
    step(pages, room=[48, 0])
    pages.length[0] = 48
    pages.block_table[0, 1] = 77
    moves = torch.empty((2, 2), dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    sv.kv_fork(pages, moves, source=dev([0, 0]), status=st)
    assert int(st.item()) == 2 and pages.block_table.cpu().tolist() == [[0, 77, 2, -1]] * 2
    assert pages.refs.cpu().tolist() == [2, 1, 2] + [0] * 5


def test_captured_on_a_stream_and_replayed():
    sv = _sv()
    pages = sv.KvPages.empty(4, 8, 40)
    cache = _pool(sv, "e4m3", 1, 2, 64, 40, 1)
    moves = torch.empty((4, 2), dtype=torch.int32, device="cuda")
    source, room = dev([0, 1, 2, 3]), dev([0] * 4)
    sv.kv_fork(pages, moves, source=source, room=room)  # (kernels set up before the capture)
    sv.kv_copy(cache, moves)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.kv_fork(pages, moves, source=source, room=room)
        sv.kv_copy(cache, moves)
        sv.kv_compact(pages, moves)
        sv.kv_copy(cache, moves)
    for src, rm, ln in (([0, 1, 2, 3], [33, 20, 0, 0], [33, 20, 0, 0]), ([1, 1, 0, -1], [21, 22, 34, 0], [21, 22, 34, 0])):
        source.copy_(dev(src)), room.copy_(dev(rm))
        f = ref.fork(*state(pages), src, None, rm)
        c = ref.compact(*f[:4], 4)
        g.replay()
        torch.cuda.synchronize()
        got = state(pages)
        assert np.array_equal(got[0], c[0]) and np.array_equal(got[3], c[1]) and np.array_equal(got[2], f[2])
        pages.length.copy_(dev(ln))


@pytest.mark.parametrize("n_seq,sources", [(1024, 32), (1024, 1), (500, 125)])
def test_many_rows_of_one_unfinished_page_each_time_alike(n_seq, sources):
    """All but one row of each source's copies its last page: counts that CTAs read while
    they are to be lowered."""
    sv = _sv()
    pages, out = (sv.KvPages.empty(n_seq, 6, 9000) for _ in range(2))
    moves = torch.empty((n_seq, 2), dtype=torch.int32, device="cuda")
    sv.kv_fork(pages, moves, room=dev([70 if s < sources else 0 for s in range(n_seq)]))
    pages.length.copy_(dev([70 if s < sources else 0 for s in range(n_seq)]))
    pages.held.copy_(dev([5 if s < sources else 0 for s in range(n_seq)]))
    source, keep = [s % sources for s in range(n_seq)], [65 + s // sources % 5 for s in range(n_seq)]
    want = step(pages, out=out, source=source, keep=keep)
    first = [t.clone() for t in (out.block_table, out.length, out.held, out.refs)]
    source, keep = dev(source), dev(keep)
    for _ in range(100):
        for t in (out.block_table, out.length, out.held, out.refs):
            t.fill_(-7)
        sv.kv_fork(pages, moves, source=source, keep=keep, out=out)
        assert np.array_equal(moves.cpu().numpy(), want)
        assert all(torch.equal(a, b) for a, b in zip(first, (out.block_table, out.length, out.held, out.refs)))


def test_the_widest_table_and_a_large_pool():
    sv = _sv()
    pages = sv.KvPages.empty(40, 4096, 400000)
    rng = random.Random(8)
    step(pages, source=[-1] * 40)
    load(pages, ref.fork(*state(pages), None, None, [rng.randrange(1, 60000) for _ in range(40)])[:4])
    pages.length.copy_(dev([min(int(h) * 16, rng.randrange(1, 60000)) for h in pages.held.tolist()]))
    step(pages, source=[rng.randrange(-1, 40) for _ in range(40)], keep=[rng.randrange(0, 65000) for _ in range(40)],
         room=[rng.randrange(0, 65536) for _ in range(40)])
