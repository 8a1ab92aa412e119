"""Refusals of the paged-cache operators, which need no GPU: the binding's
checks of tensors, and the C entry points' checks of what they are passed
(before any CUDA call)."""
import ctypes

import pytest
import torch

import greedy_speculative_decode_gb300 as sv

INVAL, NOMEM = sv.SV_E_INVAL, sv.SV_E_NOMEM


def pool(**kw):
    a = dict(format=1, n_pages=10, n_kv_heads=2, head_dim=128, scale_block=1, k=4096, v=8192, k_exp=4096, v_exp=4096)
    a.update(kw)
    return sv.SvKvPool(**a)


def rows(**kw):
    a = dict(n_seq=2, n_rows=4, max_rows=0, table_stride=5, block_table=4096, first=4096, row_start=None)
    a.update(kw)
    return sv.SvRowBatch(**a)


def write(p, r, k=4096, ks=256, v=4096, vs=256):
    return sv.lib().sv_kv_write(ctypes.byref(p), ctypes.byref(r), k, ks, v, vs, None, None)


def fetch(p, r, k=4096, ks=256, v=4096, vs=256):
    return sv.lib().sv_kv_fetch(ctypes.byref(p), ctypes.byref(r), k, ks, v, vs, None, None)


def attend(p, r, heads=4, q=4096, qs=512, out=4096, os=512, window=0, sinks=0, scale=1.0, ws=4096, n=1 << 40):
    return sv.lib().sv_attend(ctypes.byref(p), ctypes.byref(r), heads, q, qs, out, os, None, window, sinks, scale, ws, n,
                              None, None)


BAD_POOLS = [dict(format=2), dict(format=-1), dict(n_pages=0), dict(n_kv_heads=0), dict(head_dim=96), dict(head_dim=0),
             dict(scale_block=4), dict(scale_block=0), dict(k=None), dict(v=8), dict(k_exp=None), dict(v_exp=4104),
             dict(n_pages=1 << 27)]
BAD_ROWS = [dict(n_seq=0), dict(n_rows=0), dict(n_rows=5), dict(table_stride=0), dict(block_table=None), dict(first=None),
            dict(table_stride=1 << 27), dict(n_rows=1 << 29, n_seq=1)]


@pytest.mark.parametrize("call", [write, fetch, attend])
@pytest.mark.parametrize("kw", BAD_POOLS, ids=str)
def test_pools_refused(call, kw):
    assert call(pool(**kw), rows()) == INVAL


@pytest.mark.parametrize("call", [write, fetch, attend])
@pytest.mark.parametrize("kw", BAD_ROWS, ids=str)
def test_rows_refused(call, kw):
    assert call(pool(), rows(**kw)) == INVAL


@pytest.mark.parametrize("call", [write, fetch])
@pytest.mark.parametrize("kw", [dict(k=None), dict(v=None), dict(k=4104), dict(ks=128), dict(vs=260), dict(ks=-256)], ids=str)
def test_row_buffers_refused(call, kw):
    assert call(pool(), rows(), **kw) == INVAL


@pytest.mark.parametrize("kw", [dict(heads=0), dict(heads=3), dict(q=None), dict(out=None), dict(q=4098), dict(qs=504),
                                dict(os=511), dict(window=-1), dict(sinks=-1), dict(scale=float("nan")),
                                dict(scale=float("inf")), dict(ws=None), dict(ws=4112)], ids=str)
def test_attend_refused(kw):
    assert attend(pool(), rows(), **kw) == INVAL


def test_attend_limits():
    assert attend(pool(), rows(n_seq=1025, n_rows=1025)) == INVAL
    n = ctypes.c_int64()
    p, r = pool(), rows()
    assert sv.lib().sv_attend_workspace(ctypes.byref(p), ctypes.byref(r), 4, ctypes.byref(n)) == 0 and n.value > 0
    assert attend(p, r, n=n.value - 1) == NOMEM
    assert sv.lib().sv_attend_workspace(ctypes.byref(p), ctypes.byref(r), 0, ctypes.byref(n)) == INVAL
    assert sv.lib().sv_attend_workspace(None, ctypes.byref(r), 4, ctypes.byref(n)) == INVAL
    assert sv.lib().sv_attend_workspace(ctypes.byref(p), ctypes.byref(r), 4, None) == INVAL


def test_binding_refuses_host_tensors_and_wrong_shapes():
    k = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        sv.PagedKv(k, k)
    with pytest.raises(ValueError, match="shape"):
        sv.PagedKv(torch.zeros((4, 2, 8, 64), dtype=torch.bfloat16), k)
    with pytest.raises(ValueError, match="dtype"):
        sv.PagedKv(k.float(), k.float())
    with pytest.raises(ValueError, match="4-D"):
        sv.PagedKv(k[0], k[0])
    with pytest.raises(ValueError, match="CUDA"):
        sv.RowBatch(torch.zeros((2, 3), dtype=torch.int32), torch.zeros(2, dtype=torch.int32), 4)
    with pytest.raises(ValueError, match="2-D"):
        sv.RowBatch(torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), 4)
    with pytest.raises(ValueError, match="fmt"):
        sv.PagedKv.empty(4, 2, 64, fmt="int8", device="cpu")
    with pytest.raises(ValueError, match="scale_block"):
        sv.PagedKv.empty(4, 2, 64, scale_block=8, device="cpu")


@pytest.mark.parametrize("kw", [dict(window=2 ** 31), dict(sinks=2 ** 32 + 1)], ids=str)
def test_a_context_refuses_numbers_beyond_the_library_integers(kw):
    with pytest.raises(ValueError, match="at most"):
        sv.Context(None, {}, max_k=4, max_seq=64, **kw)


def test_the_workspace_does_not_grow_without_bound():
    """Long prompts: at most 512 MB; wide tables: what 64 rows need, at most 4 GB
    (or what one row does)."""
    n = ctypes.c_int64()

    def need(heads, head_dim, **kw):
        p, r = pool(head_dim=head_dim), rows(**kw)
        assert sv.lib().sv_attend_workspace(ctypes.byref(p), ctypes.byref(r), heads, ctypes.byref(n)) == 0
        return n.value

    def row(heads, head_dim, positions):  # one row's partials
        splits = min(positions, 1024) // 128 + max(0, positions - 1024) // 256
        return heads * splits * (4 * head_dim + 8)

    # small calls take what they always did
    assert need(32, 128, n_seq=32, n_rows=32, table_stride=512) == 32 * row(32, 128, 8192)
    assert need(32, 128, n_seq=32, n_rows=32, table_stride=1 << 16) == 32 * row(32, 128, 1 << 20)
    for d, stride, n_rows in ((128, 512, 8192), (128, 2048, 32768), (64, 64, 1 << 22), (256, 1 << 14, 4096), (128, 1 << 19, 77)):
        one = row(32, d, stride * 16)
        got = need(32, d, n_seq=1, n_rows=n_rows, table_stride=stride)
        assert one <= got <= max(512 << 20, min(64 * one, 4 << 30)) + 256, (d, stride, n_rows)


def test_more_query_rows_than_a_word_counts_are_refused():
    n = ctypes.c_int64()
    p, r = pool(), rows(n_seq=1, n_rows=1 << 28)
    assert sv.lib().sv_attend_workspace(ctypes.byref(p), ctypes.byref(r), 1 << 30, ctypes.byref(n)) == INVAL
    assert attend(p, r, heads=32, qs=4096, os=4096) == INVAL
