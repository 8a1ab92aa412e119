"""Refusals of the operators on pages, shared prefixes and log probabilities, which
need no GPU: the binding's checks, and the C entry points' checks of what they are
passed (before any CUDA call)."""
import ctypes

import pytest
import torch

import greedy_speculative_decode_gb300 as sv

INVAL, NOMEM = sv.SV_E_INVAL, sv.SV_E_NOMEM
L = sv.lib()
A = 4096  # an aligned address that is never read


def ref(x):
    return None if x is None else ctypes.byref(x)


def pages(**kw):
    a = dict(n_seq=3, table_stride=5, n_pages=20, block_table=A, length=2 * A, held=3 * A, refs=4 * A)
    a.update(kw)
    return sv.SvKvPages(**a)


def others(**kw):
    return pages(**{**dict(block_table=5 * A, length=6 * A, held=7 * A, refs=8 * A), **kw})


def fork(p, out=None, source=None, keep=None, room=None, moves=A, ws=A, n=1 << 40, status=None):
    return L.sv_kv_fork(ref(p), source, keep, room, ref(out), moves, ws, n, status, None)


def compact(p, out=None, moves=A, n=4, where=A, status=None):
    return L.sv_kv_compact(ref(p), ref(out), moves, n, where, status, None)


BAD_PAGES = [dict(n_seq=0), dict(n_seq=1025), dict(table_stride=0), dict(table_stride=(1 << 19) + 1), dict(n_pages=0),
             dict(n_pages=1 << 27), dict(block_table=None), dict(length=None), dict(held=None), dict(refs=None), dict(refs=A + 2)]


@pytest.mark.parametrize("call", [fork, compact])
@pytest.mark.parametrize("kw", BAD_PAGES, ids=str)
def test_tables_refused(call, kw):
    assert call(pages(**kw)) == INVAL
    assert call(pages(), others(**kw)) == INVAL
    n = ctypes.c_int64()
    assert L.sv_kv_fork_workspace(ref(pages(**kw)), ref(n)) == INVAL


@pytest.mark.parametrize("call", [fork, compact])
@pytest.mark.parametrize("kw", [dict(n_seq=2), dict(table_stride=6), dict(n_pages=21), dict(block_table=A), dict(refs=4 * A),
                                dict(length=2 * A, held=3 * A)], ids=str)
def test_results_of_other_sizes_or_in_part_in_place_refused(call, kw):
    assert call(pages(), others(**kw)) == INVAL


@pytest.mark.parametrize("kw", [dict(moves=None), dict(moves=A + 4), dict(ws=None), dict(ws=A + 8), dict(source=A + 1), dict(keep=A + 2),
                                dict(room=A + 3), dict(status=A + 1)], ids=str)
def test_fork_refused(kw):
    assert fork(pages(), **kw) == INVAL


def test_fork_workspace():
    n = ctypes.c_int64()
    assert L.sv_kv_fork_workspace(ref(pages()), ref(n)) == 0 and n.value == 4 * (20 + 15)
    assert fork(pages(), n=n.value - 1) == NOMEM
    assert L.sv_kv_fork_workspace(None, ref(n)) == INVAL and L.sv_kv_fork_workspace(ref(pages()), None) == INVAL


@pytest.mark.parametrize("kw", [dict(moves=None), dict(moves=A + 4), dict(n=0), dict(n=-1), dict(where=None), dict(where=A + 2),
                                dict(status=A + 2)], ids=str)
def test_compact_refused(kw):
    assert compact(pages(), **kw) == INVAL


def pool(**kw):
    a = dict(format=1, n_pages=10, n_kv_heads=2, head_dim=128, scale_block=1, k=A, v=A, k_exp=A, v_exp=A)
    a.update(kw)
    return sv.SvKvPool(**a)


def copy(frm, into=None, moves=A, n=3, count=None):
    a = (sv.SvKvPool * len(frm))(*frm) if frm else None
    b = (sv.SvKvPool * len(into))(*into) if into else None
    return L.sv_kv_copy(a, b, len(frm) if count is None else count, moves, n, None, None)


@pytest.mark.parametrize("kw", [dict(format=2), dict(n_pages=0), dict(n_kv_heads=0), dict(n_kv_heads=65536), dict(head_dim=96),
                                dict(scale_block=4), dict(k=None), dict(v=A + 8), dict(k_exp=None), dict(v_exp=A + 4),
                                dict(n_pages=1 << 27)], ids=str)
def test_pools_refused(kw):
    assert copy([pool(**kw)]) == INVAL
    assert copy([pool()], [pool(**kw)]) == INVAL
    assert copy([pool(), pool(**kw)]) == INVAL


@pytest.mark.parametrize("kw", [dict(format=0), dict(n_kv_heads=4), dict(head_dim=64), dict(scale_block=16), dict(n_pages=11)], ids=str)
def test_pools_that_differ_refused(kw):
    assert copy([pool(), pool(**kw)]) == INVAL
    if "n_pages" not in kw:
        assert copy([pool()], [pool(**kw)]) == INVAL
    assert copy([pool(), pool()], [pool(n_pages=30), pool(**kw)]) == INVAL


def test_moves_refused():
    assert copy([pool()], moves=None) == INVAL and copy([pool()], moves=A + 4) == INVAL
    assert copy([pool()], n=0) == INVAL and copy([pool()], count=0) == INVAL and copy([], count=1) == INVAL


# ------------------------------------------------------------------ shared prefixes
def rows(**kw):
    a = dict(n_seq=4, n_rows=8, max_rows=0, table_stride=5, block_table=A, first=A, row_start=None)
    a.update(kw)
    return sv.SvRowBatch(**a)


def prefix(**kw):
    return sv.SvSharedPrefix(**{**dict(n_groups=2, length=A, group_start=None), **kw})


def attend(p, r, x, heads=4, q=A, qs=512, out=A, os=512, scale=1.0, ws=A, n=1 << 40):
    return L.sv_attend_shared(ref(p), ref(r), ref(x), heads, q, qs, out, os, None, scale, ws, n, None, None)


@pytest.mark.parametrize("kw", [dict(n_groups=0), dict(n_groups=3), dict(n_groups=5), dict(length=None), dict(n_groups=5, group_start=A)],
                         ids=str)
def test_prefixes_refused(kw):
    n = ctypes.c_int64()
    assert attend(pool(), rows(), prefix(**kw)) == INVAL
    assert L.sv_attend_shared_workspace(ref(pool()), ref(rows()), ref(prefix(**kw)), 4, ref(n)) == INVAL


@pytest.mark.parametrize("kw", [dict(heads=0), dict(heads=3), dict(q=None), dict(out=None), dict(q=A + 2), dict(qs=504), dict(os=511),
                                dict(scale=float("nan")), dict(ws=None), dict(ws=A + 16)], ids=str)
def test_attend_shared_refused(kw):
    assert attend(pool(), rows(), prefix(), **kw) == INVAL


def test_attend_shared_limits():
    n = ctypes.c_int64()
    assert attend(pool(), rows(), None) == INVAL
    assert attend(pool(head_dim=96), rows(), prefix()) == INVAL
    assert attend(pool(), rows(n_seq=1025, n_rows=1025), prefix(n_groups=1)) == INVAL
    assert L.sv_attend_shared_workspace(ref(pool()), ref(rows()), ref(prefix()), 4, ref(n)) == 0
    assert attend(pool(), rows(), prefix(), n=n.value - 1) == NOMEM
    own = ctypes.c_int64()
    assert L.sv_attend_workspace(ref(pool()), ref(rows()), 4, ref(own)) == 0 and n.value > own.value
    assert L.sv_attend_shared_workspace(ref(pool()), ref(rows()), ref(prefix()), 4, None) == INVAL


# ------------------------------------------------------------------ log probabilities
def logprobs(x=A, dtype=0, stride=100, n=2, vocab=100, scale=1.0, tokens=A, k=1, out=A, lse=None, ent=None, top=0, tv=None, ti=None,
             status=None):
    return L.sv_logprobs(x, dtype, stride, n, vocab, scale, tokens, k, out, lse, ent, top, tv, ti, status, None)


@pytest.mark.parametrize("kw", [dict(x=None), dict(x=A + 2), dict(x=A + 1, dtype=1), dict(dtype=2), dict(dtype=-1), dict(stride=99),
                                dict(stride=-100), dict(n=0), dict(n=1 << 27), dict(vocab=0), dict(vocab=(1 << 30) + 1, stride=1 << 31),
                                dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=3e38),
                                dict(tokens=None), dict(out=None), dict(tokens=A + 1), dict(out=A + 2), dict(k=-1), dict(lse=A + 2),
                                dict(ent=A + 1), dict(top=33, tv=A), dict(top=-1), dict(top=4), dict(top=4, tv=A + 2), dict(top=4, ti=A + 1),
                                dict(status=A + 2)], ids=str)
def test_logprobs_refused(kw):
    assert logprobs(**kw) == INVAL


# ------------------------------------------------------------------ the binding
def test_binding_refuses_host_tensors_and_wrong_shapes():
    i = torch.zeros((4, 5), dtype=torch.int32)
    with pytest.raises(ValueError, match="2-D"):
        sv.KvPages(i[0], i[:, 0], i[:, 0], i[0])
    with pytest.raises(ValueError, match="1-D"):
        sv.KvPages(i, i[:, 0], i[:, 0], i)
    with pytest.raises(ValueError, match="at most"):
        sv.KvPages(torch.zeros((1025, 1), dtype=torch.int32), i[0], i[0], i[0])
    with pytest.raises(ValueError, match="CUDA"):
        sv.KvPages(i, torch.zeros(4, dtype=torch.int32), torch.zeros(4, dtype=torch.int32), torch.zeros(9, dtype=torch.int32))
    with pytest.raises(ValueError, match="1-D"):
        sv.SharedPrefix(i)
    with pytest.raises(ValueError, match="CUDA"):
        sv.SharedPrefix(torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="2-D"):
        sv.logprobs(torch.zeros(5), i, i)
    with pytest.raises(ValueError, match="CUDA"):
        sv.logprobs(torch.zeros((2, 5)), torch.zeros(2, dtype=torch.int32), torch.zeros(2))
    with pytest.raises(ValueError, match="no caches"):
        sv.KvLayers([])


# ------------------------------------------------------------------ what the header says of sizes and addresses
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("heads,n_seq,each", [(4, 4, 2), (32, 64, 1), (16, 1000, 7)])
def test_attend_shared_workspace_is_as_documented(d, heads, n_seq, each):
    r = rows(n_seq=n_seq, n_rows=n_seq * each)
    own, n = ctypes.c_int64(), ctypes.c_int64()
    assert L.sv_attend_workspace(ref(pool(head_dim=d)), ref(r), heads, ref(own)) == 0
    assert L.sv_attend_shared_workspace(ref(pool(head_dim=d)), ref(r), ref(prefix(n_groups=1)), heads, ref(n)) == 0
    row = heads * (8 * d + 16) // (2 if d == 256 else 1)
    more = n.value - own.value - row * (n_seq * each) - row * 24576 // heads
    assert 0 <= more <= 52000


@pytest.mark.parametrize("at", range(7))
def test_addresses_that_no_int32_or_float_has_are_refused(at):
    odd = [A + 2 if k == at else A for k in range(7)]
    r = rows(block_table=odd[0], first=odd[1], row_start=odd[2])
    x = prefix(length=odd[3], group_start=odd[4])
    assert L.sv_attend_shared(ref(pool()), ref(r), ref(x), 4, A, 512, A, 512, odd[5], 1.0, A, 1 << 40, odd[6], None) == INVAL
    if at not in (3, 4):
        assert L.sv_attend(ref(pool()), ref(r), 4, A, 512, A, 512, odd[5], 0, 0, 1.0, A, 1 << 40, odd[6], None) == INVAL
    if at in (0, 1, 2, 6):
        for call in (L.sv_kv_write, L.sv_kv_fetch):
            assert call(ref(pool()), ref(r), A, 512, A, 512, odd[6], None) == INVAL
