"""The paged-cache operators (kv_write, kv_fetch, attend) against the 64-bit
forms of paged_ref.py, and the properties include/sv.h promises: exact codes,
nothing touched elsewhere, results that depend on what a row sees alone."""
import numpy as np
import pytest

from . import paged_ref as ref

pytestmark = pytest.mark.gpu

PAGE = 16


def _sv():
    import greedy_speculative_decode_gb300 as sv
    return sv


def f64(t):
    return t.detach().double().cpu().numpy()


class Case:
    """A seeded pool, tables and rows on the device, and their numpy copies."""

    def __init__(self, seed, n_q, n_kv, d, lens, firsts, fmt="e4m3", block=1, ragged=True, spare=3, pages=None, back=0):
        import torch
        sv = _sv()
        g = torch.Generator().manual_seed(seed)
        self.n_q, self.n_kv, self.d, self.fmt, self.block = n_q, n_kv, d, fmt, block
        self.lens, self.firsts = lens, firsts
        n_seq, n = len(lens), sum(lens)
        width = pages or max(1, max((max(f, 0) + m + PAGE - 1) // PAGE for f, m in zip(firsts, lens)))
        total = n_seq * width + spare
        self.table_h = torch.randperm(total, generator=g)[: n_seq * width].reshape(n_seq, width).int()
        self.n_rows = n + back  # rows behind the last sequence
        x = torch.randn((2, total, n_kv, PAGE, d), generator=g) * torch.exp2(2 * torch.randn((2, total, n_kv, PAGE, 1), generator=g))
        if fmt == "bf16":
            pool = [x[0].bfloat16(), x[1].bfloat16()]
        else:
            e = torch.randint(118, 128, (2, total, n_kv, PAGE // block), generator=g)
            c = torch.randint(0, 127, (2, total, n_kv, PAGE, d), generator=g) + 128 * torch.randint(0, 2, (2, total, n_kv, PAGE, d), generator=g)
            pool = [c[0].to(torch.uint8), c[1].to(torch.uint8), e[0].to(torch.uint8), e[1].to(torch.uint8)]
        self.cache = sv.PagedKv(*[t.cuda() for t in pool])
        start = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        self.start = start.tolist()
        self.row_start = torch.from_numpy(start).cuda() if ragged or back else None
        self.table, self.first = self.table_h.cuda(), torch.tensor(firsts, dtype=torch.int32).cuda()
        self.rows = sv.RowBatch(self.table, self.first, self.n_rows, row_start=self.row_start, max_rows=max(max(lens), 1))
        self.where = ref.rows_of(firsts, self.start, self.n_rows, n_seq)
        self.g = g

    def pool_np(self):
        c = self.cache
        if self.fmt == "bf16":
            return (f64(c.k), None), (f64(c.v), None)
        return (c.k.cpu().numpy().copy(), c.k_exp.cpu().numpy().copy()), (c.v.cpu().numpy().copy(), c.v_exp.cpu().numpy().copy())

    def randn(self, *shape, spread=2.0):
        import torch
        x = torch.randn(shape, generator=self.g) * torch.exp2(spread * torch.randn(shape[:-1] + (1,), generator=self.g))
        return x.bfloat16().cuda()

    def queries(self):
        return self.randn(self.n_rows, self.n_q, self.d, spread=1.0)

    def attend(self, q, window=0, sinks=0, scale=None, **kw):
        import torch
        out = torch.full_like(q, float("nan"))
        lse = torch.full((q.shape[0], self.n_q), float("nan"), device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        _sv().attend(self.cache, self.rows, q, out, window=window, sinks=sinks, scale=scale, lse=lse, status=st, **kw)
        torch.cuda.synchronize()
        self.status = int(st.item())
        return out, lse

    def check_attend(self, window=0, sinks=0, scale=None):
        q = self.queries()
        out, lse = self.attend(q, window, sinks, scale)
        assert self.status == 0
        o, l, tol, tol_l = ref.attend(self.pool_np(), self.table_h.numpy(), self.where, f64(q), window, sinks,
                                      self.d ** -0.5 if scale is None else scale)
        n = self.start[-1]
        got, gl = f64(out)[:n], f64(lse)[:n]
        assert np.isfinite(got).all()
        over = np.abs(got - o[:n]) - tol[:n]
        assert over.max() <= 0, (over.max(), np.unravel_index(over.argmax(), over.shape))
        empty = np.isinf(l[:n])
        assert np.array_equal(np.isinf(gl), empty) and (gl[empty] < 0).all()
        assert (np.abs(gl[~empty] - l[:n][~empty]) <= tol_l[:n][~empty]).all()
        assert np.isnan(f64(out)[n:]).all() and np.isnan(f64(lse)[n:]).all()  # rows behind the last sequence
        return q, out, lse


SHAPES = [(4, 2, 64), (32, 8, 128), (8, 1, 256), (7, 1, 128), (6, 2, 64), (16, 1, 128), (20, 1, 64)]
FORMS = [("bf16", 1), ("e4m3", 1), ("e4m3", 16)]


# ------------------------------------------------------------------ write and fetch
@pytest.mark.parametrize("fmt,block", FORMS)
@pytest.mark.parametrize("n_q,n_kv,d", [(4, 2, 64), (8, 3, 128), (8, 1, 256)])
@pytest.mark.parametrize("lens,firsts", [([1], [0]), ([1], [31]), ([33], [7]), ([3, 0, 17, 1, 40], [13, 5, 0, 64, 9]),
                                         ([5, 20], [-2, -20])])
def test_write_puts_the_nearest_codes_and_nothing_else(fmt, block, n_q, n_kv, d, lens, firsts):
    import torch
    sv = _sv()
    c = Case(1, n_q, n_kv, d, lens, firsts, fmt, block, back=3)
    # rows of a fused projection: the heads of k and v lie side by side, the rows apart
    qkv = c.randn(c.n_rows, n_q + 2 * n_kv, d)
    if qkv.shape[0] > 2:
        qkv[1, n_q] = 0
        qkv[2, n_q + 1, 3] = 2.0 ** -120
    k, v = qkv[:, n_q:n_q + n_kv], qkv[:, n_q + n_kv:]
    want = c.pool_np()
    for (code, exps), x in zip(want, (k, v)):
        ref.write(code, exps, f64(x), c.table_h.numpy(), c.where)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    sv.kv_write(c.cache, c.rows, k, v, status=st)
    assert int(st.item()) == 0
    for (code, exps), (gc, ge) in zip(want, c.pool_np()):
        assert np.array_equal(code, gc)
        assert exps is None or np.array_equal(exps, ge)
    # and back: exactly the values the codes stand for
    ko = torch.full((c.n_rows, n_kv, d), 7.0, dtype=torch.bfloat16, device="cuda")
    vo = ko.clone()
    sv.kv_fetch(c.cache, c.rows, ko, vo, status=st)
    for t, (code, exps) in zip((ko, vo), want):
        got = f64(t)
        for s, r, p in c.where:
            assert np.array_equal(got[r], ref.read(code, exps, c.table_h[s, p // PAGE], p % PAGE) if p >= 0 else 0 * got[r])
        assert (got[c.start[-1]:] == 7.0).all()
    assert int(st.item()) == 0


@pytest.mark.parametrize("block", [1, 16])
def test_every_bf16_value_gets_its_nearest_code(block):
    """All finite bf16 values, each as the largest of its block, and blocks with
    an infinity or a NaN."""
    import torch
    sv = _sv()
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.uint16).view(torch.bfloat16)
    x = bits.reshape(-1, 1, 1).repeat(1, 1, 64)
    x[:, :, 1::2] *= 0.37  # others below it, rounded in every binade
    x[:, :, 5] = 0.0
    n = x.shape[0]
    width = n // PAGE
    cache = sv.PagedKv.empty(width, 1, 64, scale_block=block)
    rows = sv.RowBatch(torch.arange(width, dtype=torch.int32, device="cuda")[None], torch.zeros(1, dtype=torch.int32, device="cuda"), n)
    sv.kv_write(cache, rows, x.cuda(), x.cuda())
    code, exps = np.zeros((width, 1, PAGE, 64), np.uint8), np.zeros((width, 1, PAGE // block), np.uint8)
    xd = x.double().numpy()
    if block == 1:
        ref.write(code, exps, xd, np.arange(width)[None], ref.rows_of([0], None, n, 1))
        assert np.array_equal(cache.k.cpu().numpy(), code) and np.array_equal(cache.k_exp.cpu().numpy(), exps)
    else:
        some = list(range(0, n, 16 * 37)) + [0x7f70, 0x7f80, 0x7f90, 0xff80]
        where = [(0, r + i, r + i) for r in sorted(set(s // 16 * 16 for s in some)) for i in range(16)]
        ref.write(code, exps, xd, np.arange(width)[None], where)
        pages = sorted({p // PAGE for _, _, p in where})
        assert np.array_equal(cache.k.cpu().numpy()[pages], code[pages])
        assert np.array_equal(cache.k_exp.cpu().numpy()[pages], exps[pages])
    assert torch.equal(cache.k, cache.v) and torch.equal(cache.k_exp, cache.v_exp)
    ko = torch.empty((n, 1, 64), dtype=torch.bfloat16, device="cuda")
    vo = torch.empty_like(ko)
    sv.kv_fetch(cache, rows, ko, vo)
    bad = ~torch.isfinite(x.reshape(n, -1)).all(1)
    if block == 16:
        bad = bad.reshape(-1, 16).any(1).repeat_interleave(16)
    assert torch.isnan(ko[bad.cuda()]).all()
    fine = f64(ko)[~bad.numpy()]
    want = xd[~bad.numpy()]
    a = np.abs(want)
    if block == 1:  # half a step of the code, or of the smallest code; beyond 2^128 (1 - 2^-5) the code is 2^128
        top = a.max((1, 2), keepdims=True)
        e = np.maximum(np.ceil(np.log2(np.maximum(top, 1e-300) / 448.0)), -100)
        err = np.abs(np.minimum(np.abs(fine), 2.0 ** 128) - a)
        assert (err <= np.maximum(2.0 ** -4 * a, 2.0 ** (e - 10))).all()


def test_appending_one_by_one_gives_the_bytes_of_one_write():
    """scale_block 1: the cache does not depend on how positions were cut into calls."""
    import torch
    sv = _sv()
    a = Case(3, 8, 2, 128, [50], [0])
    k, v = a.randn(50, 2, 128), a.randn(50, 2, 128)
    sv.kv_write(a.cache, a.rows, k, v)
    b = Case(3, 8, 2, 128, [50], [0])
    first = torch.zeros(1, dtype=torch.int32, device="cuda")
    at = 0
    for n in [1, 1, 13, 1, 16, 17, 1]:
        first.fill_(at)
        sv.kv_write(b.cache, sv.RowBatch(b.table, first, n), k[at:at + n], v[at:at + n])
        at += n
    assert at == 50
    for x, y in zip(a.cache.tensors, b.cache.tensors):
        assert torch.equal(x, y)


def test_a_page_exponent_rises_with_later_rows_and_never_falls():
    import torch
    sv = _sv()
    cache = sv.PagedKv.empty(2, 1, 64, scale_block=16)
    table = torch.tensor([[1]], dtype=torch.int32, device="cuda")
    first = torch.zeros(1, dtype=torch.int32, device="cuda")
    code, exps = np.zeros((2, 1, PAGE, 64), np.uint8), np.zeros((2, 1, 1), np.uint8)
    g = torch.Generator().manual_seed(5)
    for p, size in enumerate([1.0, 0.01, 8.0, 300.0, 2.0 ** -30, 1e30, 1.0]):
        x = (size * torch.randn((1, 1, 64), generator=g)).bfloat16()
        first.fill_(p)
        sv.kv_write(cache, sv.RowBatch(table, first, 1), x.cuda(), x.cuda())
        ref.write(code, exps, x.double().numpy(), np.array([[1]]), [(0, 0, p)])
        assert np.array_equal(cache.k.cpu().numpy(), code) and np.array_equal(cache.v_exp.cpu().numpy(), exps), p
    x[0, 0, 9] = float("inf")
    first.fill_(7)
    sv.kv_write(cache, sv.RowBatch(table, first, 1), x.cuda(), x.cuda())
    assert int(cache.k_exp[1, 0, 0]) == 255 and int(cache.k[1, 0, :8].count_nonzero()) == 0
    first.fill_(0)  # its first position written again: the page starts anew
    y = torch.ones((1, 1, 64), dtype=torch.bfloat16, device="cuda")
    sv.kv_write(cache, sv.RowBatch(table, first, 1), y, y)
    assert int(cache.k_exp[1, 0, 0]) == 127 - 8


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("fmt,block", FORMS)
@pytest.mark.parametrize("n_q,n_kv,d", SHAPES)
@pytest.mark.parametrize("lens,firsts", [([1], [0]), ([1], [127]), ([4], [126]), ([3, 1, 9, 0, 2], [200, 0, 40, 7, 129])])
def test_attend(fmt, block, n_q, n_kv, d, lens, firsts):
    Case(11, n_q, n_kv, d, lens, firsts, fmt, block, back=2).check_attend()


@pytest.mark.parametrize("fmt,block", FORMS)
@pytest.mark.parametrize("n_q,n_kv,d", [(4, 2, 64), (8, 2, 128), (4, 1, 256)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (37, 3), (100, 17), (5, 300), (1000, 2)])
def test_attend_window_and_sinks(fmt, block, n_q, n_kv, d, window, sinks):
    Case(12, n_q, n_kv, d, [5, 1, 20], [290, 33, 0], fmt, block).check_attend(window, sinks)


@pytest.mark.parametrize("fmt,block", FORMS)
@pytest.mark.parametrize("n_q,n_kv,d", [(2, 1, 64), (4, 1, 128), (2, 1, 256)])
def test_attend_over_long_and_short_splits(fmt, block, n_q, n_kv, d):
    """Contexts on both sides of position 2048, where the splits get longer."""
    Case(13, n_q, n_kv, d, [3, 2, 1], [2046, 2900, 5000], fmt, block).check_attend()
    Case(14, n_q, n_kv, d, [2, 3], [5100, 2500], fmt, block).check_attend(700, 5)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("rows", [2, 5, 16, 17, 33, 130])
def test_attend_many_rows(fmt, d, rows):
    """One, two and four query tiles at a time, full and ragged."""
    Case(15, 4, 1, d, [rows, 1], [70, 3], fmt, 1).check_attend()


def test_attend_uniform_batch_and_scale():
    Case(16, 8, 2, 128, [3] * 5, [9, 0, 100, 64, 17], ragged=False).check_attend(scale=0.3)
    Case(16, 8, 2, 128, [3] * 5, [9, 0, 100, 64, 17], ragged=False).check_attend(scale=-0.05)


def test_attend_many_sequences():
    rng = np.random.default_rng(0)
    Case(17, 4, 2, 64, rng.integers(0, 3, 700).tolist(), rng.integers(0, 40, 700).tolist()).check_attend()


@pytest.mark.parametrize("fmt,block", FORMS)
def test_padding_rows_see_nothing(fmt, block):
    c = Case(18, 4, 2, 128, [3, 4, 2], [-3, -2, 10], fmt, block)
    q, out, lse = c.check_attend()
    assert (f64(out)[:5] == 0).all() and np.isneginf(f64(lse)[:5]).all()
    assert not np.isneginf(f64(lse)[5:9]).any()


@pytest.mark.parametrize("fmt,block", FORMS)
def test_the_widest_window_beside_padding_is_no_window(fmt, block):
    import torch
    c = Case(34, 4, 2, 128, [3, 4, 2], [-1, -2, 300], fmt, block)
    q = c.queries()
    want = c.attend(q)
    for window, sinks in ((2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1), (1, 2 ** 31 - 1)):
        got = c.attend(q, window, sinks)
        assert c.status == 0 and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("block", [1, 16])
@pytest.mark.parametrize("back", [1, 400])
def test_positions_of_a_zeroed_cache_are_zeros(block, back):
    """Nothing written to the last `back` positions: zero keys and values, of score 0 and weight 1."""
    import torch
    c = Case(35, 4, 2, 128, [2, 1], [410, 420], "e4m3", block)
    for s, last in enumerate((411, 420)):
        for p in range(last + 1 - back, last + 1):
            pg, sl = int(c.table_h[s, p // PAGE]), p % PAGE
            for t in c.cache.tensors[:2]:
                t[pg, :, sl] = 0
            if block == 1 or sl == 0:
                for t in c.cache.tensors[2:]:
                    t[pg, :, sl // block] = 0
    c.check_attend()
    for t in c.cache.tensors:
        t.zero_()
    q = c.queries()
    out, lse = c.attend(q)
    assert (out == 0).all()
    seen = torch.tensor([411.0, 412.0, 421.0], dtype=torch.float64)
    assert (lse.double().cpu() - seen.log()[:, None]).abs().max() <= 2.0 ** -22 * 140  # ln of sums near 2^127


def _unseen(c, window=0, sinks=0):
    """Masks [pages, 16] of the places that no row of their sequence sees."""
    import torch
    seen = torch.zeros((c.cache.n_pages, PAGE), dtype=torch.bool)
    for s, _, t in c.where:
        for p in range(t + 1):
            if window == 0 or p > t - window or p < sinks:
                seen[c.table_h[s, p // PAGE], p % PAGE] = True
    return ~seen


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 3)])
def test_what_lies_in_unseen_places_has_no_effect(fmt, d, window, sinks):
    import torch
    c = Case(19, 4, 2, d, [3, 1, 18], [45, 0, 150], fmt)
    q = c.queries()
    out, lse = c.attend(q, window, sinks)
    mask = _unseen(c, window, sinks).cuda()
    for kv, e in ((c.cache.k, c.cache.k_exp), (c.cache.v, c.cache.v_exp)):
        for pattern in range(2):
            m = mask[:, None, :, None].expand_as(kv)
            if fmt == "bf16":
                kv[m] = [float("nan"), float("-inf")][pattern]
            else:
                kv[m] = [0x7f, 0xff][pattern]
                e[mask[:, None].expand_as(e)] = [255, 0][pattern]
            out2, lse2 = c.attend(q, window, sinks)
            assert torch.equal(out, out2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_bad_value_reaches_the_rows_that_see_it_alone(fmt, d, value):
    """A draft row's infinite or NaN K or V leaves the rows before it as they are."""
    import torch
    sv = _sv()
    for which in ("k", "v"):
        c = Case(20, 4, 2, d, [6, 2], [45, 9], fmt)
        q = c.queries()
        k, v = c.randn(8, 2, d), c.randn(8, 2, d)
        sv.kv_write(c.cache, c.rows, k, v)
        out, lse = c.attend(q)
        (k if which == "k" else v)[3, 1, 5] = value  # row 3 of the first sequence, kv head 1
        sv.kv_write(c.cache, c.rows, k, v)
        out2, _ = c.attend(q)
        same = torch.ones((8, 4), dtype=torch.bool)
        same[3:6, 2:] = False
        assert torch.equal(out[same.cuda()], out2[same.cuda()])
        hit = out2[3:6, 2:].float()
        if which == "v" and fmt == "bf16":
            assert not torch.isfinite(hit[..., 5]).any()
            keep = [i for i in range(d) if i != 5]
            assert torch.equal(out[3:6, 2:, keep], out2[3:6, 2:, keep])
        elif which == "v":
            assert torch.isnan(hit).all()
        else:  # a NaN score, or one of +-infinity
            assert not torch.isfinite(hit).all() or value == float("inf")
            if value != value or fmt == "e4m3":
                assert torch.isnan(hit).all()


def test_a_bad_query_row_stays_alone():
    import torch
    for fmt in ("bf16", "e4m3"):
        c = Case(21, 4, 1, 128, [5], [60], fmt)
        q = c.queries()
        out, _ = c.attend(q)
        q[2, 1, 7] = float("nan")
        q[3, 0, 0] = float("inf")
        out2, _ = c.attend(q)
        assert torch.isnan(out2[2, 1]).all() and torch.isnan(out2[3, 0]).all()
        same = torch.ones((5, 4), dtype=torch.bool)
        same[2, 1] = same[3, 0] = False
        assert torch.equal(out[same.cuda()], out2[same.cuda()])


@pytest.mark.parametrize("size", [2.0 ** -60, 2.0 ** 60])
def test_queries_and_values_of_extreme_size(size):
    """Scores of ordinary size from tiny queries and huge keys, and values far from one."""
    import torch
    sv = _sv()
    c = Case(22, 4, 2, 128, [2], [50], "e4m3")
    n = 52
    rows = sv.RowBatch(c.table, torch.zeros(1, dtype=torch.int32, device="cuda"), n)
    k, v = c.randn(n, 2, 128, spread=0.0), c.randn(n, 2, 128, spread=4.0)
    sv.kv_write(c.cache, rows, k * size, v / size)
    q = c.queries() * (0.5 / size)
    out, lse = c.attend(q)
    o, l, tol, tol_l = ref.attend(c.pool_np(), c.table_h.numpy(), c.where, f64(q), 0, 0, 128 ** -0.5)
    assert (np.abs(f64(out) - o) <= tol).all() and (np.abs(f64(lse) - l) <= tol_l).all()


@pytest.mark.parametrize("block", [1, 16])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("rows", [1, 9])
def test_values_of_every_size_beside_one_another(block, d, rows):
    """Blocks of zeros, tiny, ordinary and huge values under scores of like size:
    each position counts in full in the denominator, whatever its values' scale."""
    import torch
    sv = _sv()
    c = Case(23, 2, 1, d, [rows], [700], "e4m3", block)
    n = 700 + rows
    every = sv.RowBatch(c.table, torch.zeros(1, dtype=torch.int32, device="cuda"), n)
    k, v = c.randn(n, 1, d, spread=0.0), c.randn(n, 1, d, spread=0.0)
    sizes = torch.tensor([0.0, 2.0 ** -98, 2.0 ** -30, 1.0, 2.0 ** 50, 2.0 ** 110])
    pick = torch.randint(0, 6, ((n + 15) // 16,), generator=c.g).repeat_interleave(16)[:n] if block == 16 else \
        torch.randint(0, 6, (n,), generator=c.g)
    pick[:130] = 0  # (the first split sees zeros alone, later ones small values first)
    v = (v.float() * sizes[pick].cuda()[:, None, None]).bfloat16()
    sv.kv_write(c.cache, every, k, v)
    for window, sinks in ((0, 0), (300, 40)):
        c.check_attend(window, sinks)


@pytest.mark.parametrize("fmt,block", FORMS)
def test_huge_keys_across_huge_queries(fmt, block):
    """Products that are zero while the scales' product is beyond fp32: scores of zero, not NaN."""
    import torch
    sv = _sv()
    c = Case(39, 2, 1, 64, [2], [40], fmt, block)
    every = sv.RowBatch(c.table, torch.zeros(1, dtype=torch.int32, device="cuda"), 42)
    k, v = c.randn(42, 1, 64, spread=0.0), c.randn(42, 1, 64, spread=0.0)
    k[:, :, :32] = 0
    k *= 2.0 ** 80
    sv.kv_write(c.cache, every, k, v)
    q = c.queries() * 2.0 ** 80
    q[:, :, 32:] = 0
    out, lse = c.attend(q)
    o, l, tol, tol_l = ref.attend(c.pool_np(), c.table_h.numpy(), c.where, f64(q), 0, 0, 0.125)
    # scores are exactly zero: an output is off by half a bf16 step, 2^-11 for each
    # weight of a mean magnitude below two, and fp32 sums of 42 terms; ln 42 by 2^-18
    assert (np.abs(f64(out) - o) <= 2.0 ** -8 * np.abs(o) + 2.0 ** -9).all() and (np.abs(f64(lse) - l) <= 2.0 ** -18).all()


# ------------------------------------------------------------------ a row's result is its own
@pytest.mark.parametrize("fmt,block", FORMS)
@pytest.mark.parametrize("n_q,n_kv,d", [(4, 2, 64), (8, 2, 128), (14, 2, 128), (8, 1, 256)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (90, 5)])
def test_rows_do_not_depend_on_the_batch(fmt, block, n_q, n_kv, d, window, sinks):
    """Every row of a ragged batch, bit for bit the same alone, as a one-row
    call, with its pages elsewhere."""
    import torch
    sv = _sv()
    c = Case(23, n_q, n_kv, d, [17, 2, 6], [2100, 300, 5], fmt, block, spare=200)
    q = c.queries()
    out, lse = c.attend(q, window, sinks)
    # the same cache on other pages
    perm = torch.randperm(c.cache.n_pages, generator=c.g).cuda()
    moved = [torch.empty_like(t) for t in c.cache.tensors]
    for a, b in zip(moved, c.cache.tensors):
        a[perm] = b
    cache2 = sv.PagedKv(*moved)
    table2 = perm[c.table.long()].int()
    for s, r, t in c.where:
        first = torch.tensor([t], dtype=torch.int32, device="cuda")
        rows = sv.RowBatch(table2[s:s + 1].contiguous(), first, 1)
        o1 = torch.empty_like(q[r:r + 1])
        l1 = torch.empty((1, n_q), device="cuda")
        sv.attend(cache2, rows, q[r:r + 1], o1, window=window, sinks=sinks, lse=l1)
        assert torch.equal(o1[0], out[r]) and torch.equal(l1[0], lse[r]), (s, r)


def test_the_same_call_twice_gives_the_same_bits():
    import torch
    c = Case(24, 32, 8, 128, [16, 3, 16, 1], [3000, 700, 2040, 4090], "e4m3")
    q = c.queries()
    out, lse = c.attend(q)
    for _ in range(20):
        o2, l2 = c.attend(q)
        assert torch.equal(out, o2) and torch.equal(lse, l2)


# ------------------------------------------------------------------ calls
def test_rows_of_a_fused_projection_and_strided_output():
    import torch
    sv = _sv()
    c = Case(25, 8, 2, 128, [4, 3], [30, 77])
    qkv = c.randn(7, 12, 128)
    q = qkv[:, :8]
    want, _ = c.attend(q.contiguous())
    wide = torch.full((7, 10, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    sv.attend(c.cache, c.rows, q, wide[:, 1:9])
    assert torch.equal(wide[:, 1:9], want)
    assert (wide[:, 0] == 3).all() and (wide[:, 9] == 3).all()


def test_bad_pages_are_passed_over_and_reported():
    import torch
    sv = _sv()
    for fmt, block in FORMS:
        c = Case(26, 4, 2, 128, [4, 4], [40, 100], fmt, block)
        q = c.queries()
        ok, _ = c.attend(q)
        before = [t.clone() for t in c.cache.tensors]
        for wrong in (-1, c.cache.n_pages, 1 << 30, -(1 << 31)):
            table = c.table.clone()
            table[1, 100 // PAGE] = wrong
            table[1, 0] = wrong
            rows = sv.RowBatch(table, c.first, 8, row_start=c.row_start, max_rows=4)
            st = torch.zeros(1, dtype=torch.int32, device="cuda")
            out = torch.empty_like(q)
            sv.attend(c.cache, rows, q, out, status=st)
            assert int(st.item()) == 2 and torch.equal(out[:4], ok[:4]) and torch.isfinite(out).all()
            k = c.randn(8, 2, 128)
            st.zero_()
            ko, vo = torch.ones_like(k), torch.ones_like(k)
            sv.kv_fetch(c.cache, rows, ko, vo, status=st)
            assert int(st.item()) == 2 and (ko[4:] == 0).all() and (vo[4:] == 0).all() and not (ko[:4] == 0).all()
            st.zero_()
            only = sv.RowBatch(table[1:].contiguous(), c.first[1:], 4)
            sv.kv_write(c.cache, only, k[:4], k[:4], status=st)
            assert int(st.item()) == 2
            assert all(torch.equal(x, y) for x, y in zip(before, c.cache.tensors))
        # a position that the table does not reach
        rows = sv.RowBatch(c.table[:, :3].contiguous(), c.first, 8, row_start=c.row_start, max_rows=4)
        st.zero_()
        sv.attend(c.cache, rows, q, out, status=st)
        assert int(st.item()) == 2 and torch.equal(out[:4], ok[:4]) and torch.isfinite(out).all()
        far = torch.tensor([40, (1 << 31) - 1], dtype=torch.int32, device="cuda")
        rows = sv.RowBatch(c.table, far, 8, row_start=c.row_start, max_rows=4)
        st.zero_()
        sv.attend(c.cache, rows, q, out, status=st, window=30)
        sv.kv_write(c.cache, sv.RowBatch(c.table[1:].contiguous(), far[1:], 4), k[:4], k[:4])
        assert int(st.item()) == 2 and torch.isfinite(out).all()
        assert all(torch.equal(x, y) for x, y in zip(before, c.cache.tensors))


def test_row_starts_outside_the_buffers_touch_nothing_outside():
    import torch
    sv = _sv()
    c = Case(27, 4, 2, 64, [2, 3], [20, 30])
    q = c.queries()
    out = torch.full((9, 4, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    starts = torch.tensor([-4, 2, 4000], dtype=torch.int32, device="cuda")
    rows = sv.RowBatch(c.table, c.first, 5, row_start=starts)
    sv.attend(c.cache, rows, q, out[2:7])
    torch.cuda.synchronize()
    assert (out[:2] == 5).all() and (out[7:] == 5).all()


@pytest.mark.parametrize("starts", [[0, 5, 2, 5], [3, 0, 5, 5], [5, 4, 3, 0], [0, 2, 1, 5]])
def test_row_starts_that_decrease_touch_nothing_outside(starts):
    import torch
    sv = _sv()
    for fmt, block in FORMS:
        c = Case(36, 4, 2, 64, [2, 2, 1], [20, 30, 3], fmt, block)
        out = torch.full((9, 4, 64), 5.0, dtype=torch.bfloat16, device="cuda")
        rows = sv.RowBatch(c.table, c.first, 5, row_start=torch.tensor(starts, dtype=torch.int32, device="cuda"))
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        sv.attend(c.cache, rows, c.queries(), out[2:7], status=st)
        torch.cuda.synchronize()
        assert (out[:2] == 5).all() and (out[7:] == 5).all() and int(st.item()) == 2


def test_captured_and_replayed_with_other_lengths():
    """A graph of write and attend, replayed while the program advances the
    lengths on the device: each replay as the eager calls."""
    import torch
    sv = _sv()
    c = Case(28, 8, 2, 128, [2, 2, 2], [0, 0, 0], pages=20)
    first = torch.tensor([5, 130, 61], dtype=torch.int32, device="cuda")
    rows = sv.RowBatch(c.table, first, 6)
    q, k, v = c.randn(6, 8, 128), c.randn(6, 2, 128), c.randn(6, 2, 128)
    out = torch.empty_like(q)
    s = torch.cuda.Stream()
    ws = torch.empty(sv.attend_workspace(c.cache, rows, 8), dtype=torch.uint8, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        sv.attend(c.cache, rows, q, out, workspace=ws)  # sets the kernels' attributes
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        sv.kv_write(c.cache, rows, k, v)
        sv.attend(c.cache, rows, q, out, workspace=ws)
        first.add_(2)
    twin = sv.PagedKv(*[t.clone() for t in c.cache.tensors])
    at = [5, 130, 61]
    for step in range(6):
        for x in (q, k, v):
            x.copy_(c.randn(*x.shape))
        g.replay()
        torch.cuda.synchronize()
        f = torch.tensor([a + 2 * step for a in at], dtype=torch.int32, device="cuda")
        r = sv.RowBatch(c.table, f, 6)
        o = torch.empty_like(q)
        sv.kv_write(twin, r, k, v)
        sv.attend(twin, r, q, o)
        assert torch.equal(o, out)
        assert all(torch.equal(x, y) for x, y in zip(twin.tensors, c.cache.tensors))


def test_two_graphs_of_one_batch_replayed_at_once():
    """Graphs captured without a workspace of the caller's share none, so they
    may be replayed beside one another."""
    import torch
    sv = _sv()
    c = Case(32, 32, 8, 128, [4] * 8, [3000] * 8)
    qs, want, outs, graphs = [c.queries() for _ in range(2)], [], [], []
    for q in qs:
        want.append(c.attend(q)[0])
    streams = [torch.cuda.Stream() for _ in qs]
    for q, s in zip(qs, streams):
        out = torch.empty_like(q)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            for _ in range(5):
                sv.attend(c.cache, c.rows, q, out)
        outs.append(out)
        graphs.append(g)
    for _ in range(10):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_one_batch_on_two_streams_at_once():
    import torch
    sv = _sv()
    c = Case(33, 32, 8, 128, [4] * 8, [3000] * 8)
    qs = [c.queries() for _ in range(2)]
    want = [c.attend(q)[0] for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    outs = [torch.empty_like(q) for q in qs]
    torch.cuda.synchronize()
    for i in range(20):
        for q, o, s in zip(qs, outs, streams):
            if i % 2:
                sv.attend(c.cache, c.rows, q, o, stream=s)
            else:
                with torch.cuda.stream(s):
                    sv.attend(c.cache, c.rows, q, o)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_one_batch_of_two_threads_on_one_stream():
    import threading
    import torch
    sv = _sv()
    c = Case(37, 8, 2, 128, [2] * 4, [500] * 4)
    qs = [c.queries() for _ in range(2)]
    want = [c.attend(q)[0] for q in qs]
    outs = [[torch.empty_like(q) for _ in range(300)] for q in qs]
    meet = threading.Barrier(2)

    def work(q, o):
        meet.wait()
        for x in o:
            sv.attend(c.cache, c.rows, q, x)

    threads = [threading.Thread(target=work, args=a) for a in zip(qs, outs)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    assert all(torch.equal(x, w) for o, w in zip(outs, want) for x in o)


def test_numbers_beyond_the_library_integers_are_refused():
    """ctypes would drop their upper bits."""
    sv = _sv()
    c = Case(38, 2, 1, 64, [1], [3])
    q = c.queries()
    for kw in (dict(window=2 ** 32), dict(sinks=2 ** 32 + 4), dict(window=2 ** 31), dict(sinks=-2 ** 32)):
        with pytest.raises(ValueError, match="must not be negative, nor above"):
            c.attend(q, **kw)
    with pytest.raises(ValueError, match="n_rows"):
        sv.RowBatch(c.table, c.first, 2 ** 32 + 1)
    with pytest.raises(ValueError, match="max_rows"):
        sv.RowBatch(c.table, c.first, 1, max_rows=2 ** 32)


def test_calls_on_two_streams_at_once():
    import torch
    a, b = Case(29, 32, 8, 128, [4] * 8, [3000] * 8), Case(30, 32, 8, 128, [1] * 20, [1500] * 20)
    qa, qb = a.queries(), b.queries()
    wa, wb = a.attend(qa)[0], b.attend(qb)[0]
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    oa, ob = [torch.empty_like(wa) for _ in range(10)], [torch.empty_like(wb) for _ in range(10)]
    torch.cuda.synchronize()
    for i in range(10):
        with torch.cuda.stream(sa):
            _sv().attend(a.cache, a.rows, qa, oa[i])
        with torch.cuda.stream(sb):
            _sv().attend(b.cache, b.rows, qb, ob[i])
    torch.cuda.synchronize()
    assert all(torch.equal(wa, x) for x in oa) and all(torch.equal(wb, x) for x in ob)


def test_pools_beyond_four_gigabytes():
    """Pages whose codes lie more than 2^32 bytes into the pool."""
    import torch
    sv = _sv()
    n_pages = (1 << 32) // (8 * PAGE * 128) + 40
    cache = sv.PagedKv.empty(n_pages, 8, 128)
    table = torch.tensor([[n_pages - 1, 3, n_pages - 20]], dtype=torch.int32, device="cuda")
    first = torch.zeros(1, dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(6)
    k, v, q = (torch.randn((40, h, 128), generator=g).bfloat16().cuda() for h in (8, 8, 32))
    rows = sv.RowBatch(table, first, 40)
    sv.kv_write(cache, rows, k, v)
    out = torch.empty_like(q)
    sv.attend(cache, rows, q, out)
    small = sv.PagedKv.empty(3, 8, 128)
    srows = sv.RowBatch(torch.tensor([[0, 1, 2]], dtype=torch.int32, device="cuda"), first, 40)
    sv.kv_write(small, srows, k, v)
    want = torch.empty_like(q)
    sv.attend(small, srows, q, want)
    assert torch.equal(out, want) and torch.equal(small.k, cache.k[table[0].long()])
    ko, vo = torch.empty_like(k), torch.empty_like(k)
    ks, vs = torch.empty_like(k), torch.empty_like(k)
    sv.kv_fetch(cache, rows, ko, vo)
    sv.kv_fetch(small, srows, ks, vs)
    assert torch.equal(ko, ks) and torch.equal(vo, vs)


def test_prefix_pages_shared_by_sequences():
    import torch
    sv = _sv()
    c = Case(31, 8, 2, 128, [1, 1], [40, 44])
    table = c.table.clone()
    table[1, :2] = table[0, :2]  # positions 0 .. 31 are common
    rows = sv.RowBatch(table, c.first, 2)
    q = c.queries()
    out = torch.empty_like(q)
    sv.attend(c.cache, rows, q, out)
    for s in range(2):
        o = torch.empty_like(q[:1])
        sv.attend(c.cache, sv.RowBatch(table[s:s + 1].contiguous(), c.first[s:s + 1], 1), q[s:s + 1], o)
        assert torch.equal(o[0], out[s])


def test_a_decode_loop_written_read_and_attended():
    """Prompt, steps of one and of several rows, a rollback: the operators as a
    program runs them, against the 64-bit form over the values it wrote."""
    import torch
    sv = _sv()
    for fmt, block in FORMS:
        n_q, n_kv, d = 8, 2, 128
        cache = sv.PagedKv.empty(12, n_kv, d, fmt=fmt, scale_block=block)
        table_h = torch.randperm(12, generator=torch.Generator().manual_seed(7)).int()[None]
        table = table_h.cuda()
        pool = ((np.zeros(cache.k.shape) if fmt == "bf16" else np.zeros(cache.k.shape, np.uint8),
                 None if fmt == "bf16" else np.zeros(cache.k_exp.shape, np.uint8)) for _ in range(2))
        pool = tuple(pool)
        g = torch.Generator().manual_seed(8)
        length = 0
        for n, keep in [(70, 70), (1, 1), (4, 2), (1, 1), (8, 8), (16, 3), (1, 1)]:
            q, k, v = ((torch.randn((n, h, d), generator=g) * 2).bfloat16() for h in (n_q, n_kv, n_kv))
            rows = sv.RowBatch(table, torch.tensor([length], dtype=torch.int32, device="cuda"), n)
            out = torch.empty((n, n_q, d), dtype=torch.bfloat16, device="cuda")
            sv.kv_write(cache, rows, k.cuda(), v.cuda())
            sv.attend(cache, rows, q.cuda(), out)
            where = [(0, i, length + i) for i in range(n)]
            for (code, exps), x in zip(pool, (k, v)):
                ref.write(code, exps, f64(x), table_h.numpy(), where)
            o, _, tol, _ = ref.attend(pool, table_h.numpy(), where, f64(q), 0, 0, d ** -0.5)
            assert (np.abs(f64(out) - o) <= tol).all()
            length += keep


@pytest.mark.parametrize("fmt,d", [("e4m3", 128), ("bf16", 64), ("bf16", 256)])
@pytest.mark.parametrize("lens,firsts,window,sinks", [([300], [0], 0, 0), ([150, 150, 150], [500, 0, 700], 60, 2),
                                                      ([140] * 6, [-100, -137, -90, -50, -120, -139], 0, 0)],
                         ids=["prompt", "window", "padding"])
def test_runs_of_ctas_that_begin_in_places_their_tile_does_not_see(fmt, d, lens, firsts, window, sinks):
    """More chunks than there are CTAs, so that runs of work begin in the middle
    of a tile's list: among chunks behind an early tile's rows, in front of a
    late tile's window, or in a tile of padding alone.  The tiles that follow in
    the same run keep their own queries, call after call."""
    import torch
    n_q, n_kv = (32, 8) if d < 256 else (16, 4)
    c = Case(40, n_q, n_kv, d, lens, firsts, fmt)
    q, out, lse = c.check_attend(window, sinks)
    for _ in range(60):
        o2, l2 = c.attend(q, window, sinks)
        assert torch.equal(out, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("n_q,n_kv,d", [(4, 2, 64), (4, 2, 128), (4, 1, 256)])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_an_infinite_value_is_the_same_in_every_batch(n_q, n_kv, d, value):
    """Position 5 lies in a page that the row at 20 sees whole, and that a tile
    which begins at 2 does not.  Weights are like in size, so that the weighted
    sum of an infinity is that infinity."""
    import torch
    sv = _sv()
    c = Case(41, n_q, n_kv, d, [25, 3, 2], [2, 300, 1500], "bf16")
    for s, p in ((0, 5), (1, 281), (2, 130), (2, 700), (2, 1100), (2, 1101), (2, 1490)):  # several splits of one run
        c.cache.v[int(c.table_h[s, p // PAGE]), 0, p % PAGE, 7] = value
    q = c.queries()
    out, lse = c.attend(q, scale=0.02)
    hit = out[:, :n_q // n_kv, 7]
    assert torch.isfinite(hit[:3]).all()  # positions 2 .. 4
    same = torch.isnan(hit[3:]) if value != value else hit[3:] == value
    assert same.all()
    rest = out.clone()
    rest[3:, :n_q // n_kv, 7] = 0
    assert torch.isfinite(rest).all()
    for s, r, t in c.where:
        o1, l1 = torch.empty_like(q[:1]), torch.empty((1, n_q), device="cuda")
        rows = sv.RowBatch(c.table[s:s + 1], torch.tensor([t], dtype=torch.int32, device="cuda"), 1)
        sv.attend(c.cache, rows, q[r:r + 1], o1, scale=0.02, lse=l1)
        assert torch.equal(o1[0].view(torch.int16), out[r].view(torch.int16)) and torch.equal(l1[0], lse[r]), t


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("rows", [1, 9, 40])
@pytest.mark.parametrize("size", [2.0 ** 117, 2.0 ** -100])
def test_bf16_values_near_the_ends_of_their_range(d, rows, size):
    """A mean of finite values is finite, where the sum of thousands of them is not."""
    n_q = 32 if rows == 40 else 2  # (the merge's other form)
    c = Case(42, n_q, 2, d, [rows, 1], [3500, 40], "bf16")
    x = c.randn(c.cache.n_pages, 2, PAGE, d, spread=0.0).float().clamp(-3.9, 3.9)
    c.cache.v.copy_((x.abs() * size).bfloat16())
    c.check_attend(scale=1e-4)
    c.cache.v.copy_((x * size).bfloat16())
    c.check_attend(scale=1e-4)


def _pieces(c, q, lens, firsts, window, sinks, k_rows):
    """Every sequence by itself, k_rows rows a call, on a table cut to what they need."""
    import torch
    sv = _sv()
    out, lse = torch.zeros_like(q), torch.zeros((q.shape[0], q.shape[1]), device="cuda")
    at = 0
    for s, (n, f) in enumerate(zip(lens, firsts)):
        for i in range(0, n, k_rows):
            m = min(k_rows, n - i)
            pages = max(1, (f + i + m + PAGE - 1) // PAGE)
            first = torch.tensor([f + i], dtype=torch.int32, device="cuda")
            rows = sv.RowBatch(c.table[s:s + 1, :pages].contiguous(), first, m)
            sl = slice(at + i, at + i + m)
            o, l = torch.empty_like(q[sl]), torch.empty_like(lse[sl])
            sv.attend(c.cache, rows, q[sl], o, window=window, sinks=sinks, lse=l)
            out[sl], lse[sl] = o, l
        at += n
    return out, lse


@pytest.mark.parametrize("fmt,window,sinks", [("e4m3", 0, 0), ("bf16", 70, 3)])
def test_calls_of_many_rows_are_taken_in_blocks(fmt, window, sinks):
    """A table for 65536 positions: 300 rows of 32 heads would have 1.3 GB of
    partials.  The blocks' borders fall inside sequences; nothing behind the
    workspace is written; captured and replayed the same."""
    import torch
    sv = _sv()
    lens, firsts = [90, 0, 1, 100, 3, 104], [200, 9, 700, -20, 31, 0]
    c = Case(43, 32, 2, 128, lens, firsts, fmt, back=2)
    table = torch.full((len(lens), 4096), -1, dtype=torch.int32, device="cuda")
    table[:, :c.table.shape[1]] = c.table
    rows = sv.RowBatch(table, c.first, c.n_rows, row_start=c.row_start)
    q = c.queries()
    need = sv.attend_workspace(c.cache, rows, 32)
    assert need <= 512 << 20
    ws = torch.full((need + 4096,), 0x5a, dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = torch.full_like(q, 7.0), torch.full((c.n_rows, 32), 7.0, device="cuda")
    kw = dict(window=window, sinks=sinks, lse=lse, status=st)
    sv.attend(c.cache, rows, q, out, workspace=ws[:need], **kw)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and (ws[need:] == 0x5a).all()
    n = sum(lens)
    assert (out[n:] == 7).all() and (lse[n:] == 7).all()
    want, want_l = _pieces(c, q, lens, firsts, window, sinks, 16)
    assert torch.equal(out[:n], want[:n]) and torch.equal(lse[:n], want_l[:n])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.attend(c.cache, rows, q, out, **kw)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[:n], want[:n])
    # in the place of the queries
    sv.attend(c.cache, rows, q, q, **kw)
    assert torch.equal(q[:n], want[:n])


def test_blocks_of_rows_far_beyond_the_table():
    """Rows at 2^30 and more, whose windows reach back to positions that differ
    from row to row: the blocks' border elsewhere."""
    import torch
    sv = _sv()
    c = Case(48, 32, 1, 128, [300], [0], "e4m3")
    table = torch.full((1, 4096), -1, dtype=torch.int32, device="cuda")
    table[:, :c.table.shape[1]] = c.table
    far = torch.tensor([1 << 30], dtype=torch.int32, device="cuda")
    q = c.queries()
    window = (1 << 30) + 40  # row i sees the positions above i - 40
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    sv.attend(c.cache, sv.RowBatch(table, far, 300), q, out, window=window, status=st)
    assert int(st.item()) == 2  # the table does not reach them
    # (a sequence begins at 2^30 at most, so fewer rows instead of later ones)
    some = sv.RowBatch(table, far, 124)
    assert sv.attend_workspace(c.cache, some, 32) > sv.attend_workspace(c.cache, sv.RowBatch(table, far, 300), 32)
    o = torch.empty_like(q[:124])
    sv.attend(c.cache, some, q[:124], o, window=window)
    assert torch.equal(o, out[:124])


@pytest.mark.parametrize("ragged", [True, False])
def test_long_prompts_in_blocks(ragged):
    """2000 rows of two sequences, three blocks, against calls of 64 rows."""
    import torch
    sv = _sv()
    lens, firsts = [1000, 1000], [0, 37]
    c = Case(44, 32, 8, 128, lens, firsts, "e4m3", pages=1100, ragged=ragged)
    assert sv.attend_workspace(c.cache, c.rows, 32) <= 512 << 20
    q = c.queries()
    out, lse = c.attend(q)
    want, want_l = _pieces(c, q, lens, firsts, 0, 0, 64)
    assert torch.equal(out, want) and torch.equal(lse, want_l)


@pytest.mark.parametrize("fmt,block", FORMS)
@pytest.mark.parametrize("n_q,n_kv,d", [(4, 1, 64), (8, 2, 128), (4, 1, 256)])
def test_attend_where_the_splits_get_longer(fmt, block, n_q, n_kv, d):
    """Rows, window edges and sinks on both sides of position 1024, one by one."""
    for first, lens in ((1020, 9), (1023, 1), (1024, 1), (1278, 4)):
        c = Case(45, n_q, n_kv, d, [lens, 2], [first, 1022], fmt, block)
        c.check_attend()
        for window, sinks in ((1, 0), (2, 1024), (3, 1025), (257, 1023), (900, 2)):
            c.check_attend(window, sinks)
    for t in (1030, 1500):  # windows that begin at 1022 .. 1026
        c = Case(46, n_q, n_kv, d, [1, 1, 1], [t, t + 1, t - 1], fmt, block)
        for lo in (1022, 1023, 1024, 1025, 1026):
            c.check_attend(t - lo + 1, 3)


@pytest.mark.parametrize("fmt,block", FORMS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 4), (300, 200)])
def test_attend_more_chunks_than_ctas(fmt, block, window, sinks):
    """CTAs begin in the middle of a tile's list and go on into other tiles, kv
    heads and sequences, empty ones among them."""
    c = Case(47, 32, 16, 64, [70, 0, 33, 1, 0, 90, 41], [300, 5, 0, 1100, 77, 150, -30], fmt, block, back=3)
    q, out, lse = c.check_attend(window, sinks)
    import torch
    for _ in range(20):
        o2, l2 = c.attend(q, window, sinks)
        n = c.start[-1]
        assert torch.equal(out[:n], o2[:n]) and torch.equal(lse[:n], l2[:n])
