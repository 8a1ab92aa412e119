"""Python binding of libsv.so: argument marshalling over the C-ABI only.

Every step of decode / verify runs in the library's CUDA kernels; this module
passes pointers and sizes. PyTorch provides device memory and streams. If
the compiled library is missing the import fails: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsv.so")

SV_OK, SV_E_INVAL, SV_E_NOMEM, SV_E_CUDA, SV_E_STATE = 0, -1, -2, -3, -4
SV_LIN_O, SV_LIN_GATE_UP, SV_LIN_DOWN, SV_LIN_LM_HEAD = 1, 2, 3, 4
PAGE_SIZE = 16
MAX_K = 32
MAX_PREFILL_ROWS = 128
SV_KV_BF16, SV_KV_E4M3 = 0, 1
ATTEND_MAX_SEQ = 1024
_INT_MAX = 2 ** 31 - 1
_ERRNAMES = {SV_E_INVAL: "SV_E_INVAL", SV_E_NOMEM: "SV_E_NOMEM", SV_E_CUDA: "SV_E_CUDA",
             SV_E_STATE: "SV_E_STATE"}

_P = ctypes.c_void_p
_PP = ctypes.POINTER(ctypes.c_void_p)
_i32 = ctypes.c_int32


class SvConfig(ctypes.Structure):
    _fields_ = [(n, _i32) for n in ("n_layers", "hidden", "n_q_heads", "n_kv_heads", "head_dim",
                                   "ffn", "vocab")] + [
        ("rms_eps", ctypes.c_float), ("rope_theta", ctypes.c_float)] + [
        (n, _i32) for n in ("qk_norm", "act", "tie_embeddings", "page_size", "max_pages", "max_k",
                            "max_seq", "kv_delayed", "kv_format", "window", "sinks")]


LAYER_KEYS = ("attn_norm", "wqkv", "q_norm", "k_norm", "wo", "ffn_norm", "w_gate_up", "w_down")


class SvWeights(ctypes.Structure):
    _fields_ = [("embed", _P), ("lm_head", _P), ("final_norm", _P)] + [(k, _PP) for k in LAYER_KEYS]


class SvKvPool(ctypes.Structure):
    _fields_ = [(n, _i32) for n in ("format", "n_pages", "n_kv_heads", "head_dim", "scale_block")] + [
        (n, _P) for n in ("k", "v", "k_exp", "v_exp")]


class SvRowBatch(ctypes.Structure):
    _fields_ = [(n, _i32) for n in ("n_seq", "n_rows", "max_rows", "table_stride")] + [
        (n, _P) for n in ("block_table", "first", "row_start")]


class SvError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{_ERRNAMES.get(code, code)}: {msg}")
        self.code = code


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build() (needs nvcc)")
    L = ctypes.CDLL(LIB_PATH)
    L.sv_create.argtypes = [ctypes.POINTER(SvConfig), ctypes.POINTER(SvWeights), _P, ctypes.POINTER(_P)]
    L.sv_destroy.argtypes = [_P]
    L.sv_destroy.restype = None
    L.sv_prefill.argtypes = [_P, _P, _i32, _P, _P]
    L.sv_decode.argtypes = [_P, _i32, _P, _P]
    L.sv_verify.argtypes = [_P, _P, _i32, _P, _P, _P]
    L.sv_verify_async.argtypes = [_P, _P, _i32, _P, _P]
    L.sv_reserve.argtypes = [_P, _i32]
    L.sv_sync.argtypes = [_P]
    L.sv_truncate.argtypes = [_P, _i32]
    L.sv_seq_len.argtypes = [_P]
    L.sv_kv_read.argtypes = [_P, _i32, _i32, _i32, _P, _P]
    L.sv_shuffle_pages.argtypes = [_P, ctypes.c_uint64]
    L.sv_trace_hidden.argtypes = [_P, _P, _i32]
    L.sv_step_kernel_count.argtypes = [_P, _i32, _i32]
    L.sv_prefill_blocks.argtypes = [_i32, _i32, _P, _i32]
    L.sv_spec_generate.argtypes = [_P, _P, _i32, _i32, _i32, _P, _P, _P, _P]
    L.sv_time_linear.argtypes = [_P, _i32, _i32, _i32, ctypes.POINTER(ctypes.c_float),
                                 ctypes.POINTER(ctypes.c_double)]
    L.sv_lm_head_noalloc.argtypes = [_P, _P, _P, _i32, _i32, _i32, ctypes.c_float, _P, _P, _P, _P]
    i64 = ctypes.c_int64
    L.sv_kv_write.argtypes = L.sv_kv_fetch.argtypes = [_P, _P, _P, i64, _P, i64, _P, _P]
    L.sv_attend_workspace.argtypes = [_P, _P, _i32, ctypes.POINTER(i64)]
    L.sv_attend.argtypes = [_P, _P, _i32, _P, i64, _P, i64, _P, _i32, _i32, ctypes.c_float, _P, i64, _P, _P]
    L.sv_last_error.argtypes = [_P]
    L.sv_last_error.restype = ctypes.c_char_p
    for name in ("sv_create", "sv_prefill", "sv_decode", "sv_verify", "sv_verify_async",
                 "sv_reserve", "sv_sync", "sv_truncate", "sv_seq_len", "sv_kv_read",
                 "sv_shuffle_pages", "sv_trace_hidden", "sv_step_kernel_count", "sv_time_linear",
                 "sv_lm_head_noalloc", "sv_prefill_blocks", "sv_kv_write", "sv_kv_fetch",
                 "sv_attend_workspace", "sv_attend"):
        getattr(L, name).restype = _i32
    return L


_lib = _load()


def lib():
    return _lib


def _i32_array(vals):
    vals = [int(v) for v in vals]
    return (ctypes.c_int32 * len(vals))(*vals)


def _ptr(t) -> int:
    return 0 if t is None else int(t.data_ptr())


def _check_tensor(t, name, dtype, shape):
    """The C call takes raw pointers and cannot check what they point to: a
    wrong dtype, shape, device or layout here would become out-of-bounds
    device accesses there."""
    if t is None:
        return
    if not getattr(t, "is_cuda", False):
        raise ValueError(f"{name}: must be a CUDA tensor")
    if str(t.dtype) != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")


def _check_buf(t, name, dtype, min_numel, cuda=False):
    """A buffer that a step's kernels read or write whole (tokens, result,
    logits): the C call sees only its address, so a buffer of another type,
    not contiguous or too small would become out-of-bounds accesses there.
    cuda: must also be device memory (the library checks the asynchronous
    call's token and result buffers itself)."""
    if t is None:
        return
    if cuda and not getattr(t, "is_cuda", False):
        raise ValueError(f"{name}: must be a CUDA tensor")
    if str(t.dtype) != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if t.numel() < min_numel:
        raise ValueError(f"{name}: {t.numel()} elements, at least {min_numel} needed")


def lm_head_noalloc(x, gain, w, logits, argmax=None, status=None, eps=1e-6, stream=None):
    """sv_lm_head_noalloc: logits and greedy tokens of M rows without any
    device allocation by the library (scratch is a fixed array inside it).
    x: bf16 [M, hidden]; gain: bf16 [hidden]; w: bf16 [vocab, hidden];
    logits: fp32 [M, vocab]; argmax: int32 [M] or None; status: int32 [1] or
    None. All CUDA tensors owned by the caller, contiguous. Asynchronous on
    `stream`. Raises ValueError before any device work if a tensor does not
    match these shapes and types."""
    if getattr(x, "dim", lambda: 0)() != 2 or getattr(w, "dim", lambda: 0)() != 2:
        raise ValueError("x and w must be 2-D tensors")
    M, hidden = int(x.shape[0]), int(x.shape[1])
    vocab = int(w.shape[0])
    _check_tensor(x, "x", "torch.bfloat16", (M, hidden))
    _check_tensor(gain, "gain", "torch.bfloat16", (hidden,))
    _check_tensor(w, "w", "torch.bfloat16", (vocab, hidden))
    _check_tensor(logits, "logits", "torch.float32", (M, vocab))
    _check_tensor(argmax, "argmax", "torch.int32", (M,))
    _check_tensor(status, "status", "torch.int32", (1,))
    s = _P(stream.cuda_stream) if stream is not None else _P(0)
    rc = _lib.sv_lm_head_noalloc(_P(_ptr(x)), _P(_ptr(gain)), _P(_ptr(w)), M, hidden, vocab,
                                 float(eps), _P(_ptr(logits)), _P(_ptr(argmax)), _P(_ptr(status)), s)
    if rc != SV_OK:
        raise SvError(rc, "sv_lm_head_noalloc rejected the shapes (scratch limit 8 MiB, "
                          "1 <= M <= 32, hidden % 128 == 0) or a CUDA call failed")


class PagedKv:
    """A paged K/V cache of the caller's tensors (sv_kv_pool in include/sv.h).

    k, v: codes [n_pages, n_kv_heads, 16, head_dim], bf16, or uint8 holding
    e4m3 codes; then k_exp, v_exp: uint8 exponent bytes [n_pages, n_kv_heads,
    16 / scale_block], scale_block 1 or 16. All contiguous on one CUDA device,
    kept alive by this object. PagedKv.empty allocates them."""

    def __init__(self, k, v, k_exp=None, v_exp=None):
        if getattr(k, "dim", lambda: 0)() != 4:
            raise ValueError("k: must be a 4-D tensor [n_pages, n_kv_heads, 16, head_dim]")
        n_pages, n_kv, page, d = (int(x) for x in k.shape)
        if page != PAGE_SIZE or d not in (64, 128, 256) or n_pages < 1 or n_kv < 1:
            raise ValueError(f"k: shape {tuple(k.shape)}, expected [n_pages, n_kv_heads, 16, 64 | 128 | 256]")
        kind = str(k.dtype)
        if kind not in ("torch.bfloat16", "torch.uint8"):
            raise ValueError(f"k: dtype {k.dtype}, expected torch.bfloat16 or torch.uint8 (e4m3 codes)")
        self.format = SV_KV_BF16 if kind == "torch.bfloat16" else SV_KV_E4M3
        _check_tensor(k, "k", kind, k.shape)
        _check_tensor(v, "v", kind, k.shape)
        self.scale_block = 1
        if self.format == SV_KV_E4M3:
            if k_exp is None or v_exp is None:
                raise ValueError("an 8-bit cache needs k_exp and v_exp")
            per = int(k_exp.shape[-1]) if k_exp.dim() == 3 else 0
            if per not in (1, PAGE_SIZE):
                raise ValueError(f"k_exp: shape {tuple(k_exp.shape)}, expected [n_pages, n_kv_heads, 16 or 1]")
            self.scale_block = PAGE_SIZE // per
            _check_tensor(k_exp, "k_exp", "torch.uint8", (n_pages, n_kv, per))
            _check_tensor(v_exp, "v_exp", "torch.uint8", (n_pages, n_kv, per))
        elif k_exp is not None or v_exp is not None:
            raise ValueError("a bf16 cache takes no exponents")
        self.tensors = tuple(t for t in (k, v, k_exp, v_exp) if t is not None)
        for t in self.tensors:
            if t.device != k.device:
                raise ValueError("the cache's tensors lie on different devices")
            if t.data_ptr() % 16:
                raise ValueError("the cache's tensors must be aligned to 16 bytes")
        import torch
        self._bf16, self._torch = torch.bfloat16, torch._C  # (at hand: looked up on every call)
        self.k, self.v, self.k_exp, self.v_exp = k, v, k_exp, v_exp
        self.n_pages, self.n_kv_heads, self.head_dim, self.device = n_pages, n_kv, d, k.device
        self._index = k.device.index
        self._c = SvKvPool(self.format, n_pages, n_kv, d, self.scale_block, _ptr(k), _ptr(v), _ptr(k_exp),
                           _ptr(v_exp))
        self._p = ctypes.byref(self._c)

    @classmethod
    def empty(cls, n_pages: int, n_kv_heads: int, head_dim: int, *, fmt: str = "e4m3", scale_block: int = 1,
              device="cuda"):
        """A zeroed cache; fmt "e4m3" or "bf16"."""
        import torch
        if fmt not in ("e4m3", "bf16"):
            raise ValueError(f"fmt {fmt!r}, expected 'e4m3' or 'bf16'")
        if scale_block not in (1, PAGE_SIZE):
            raise ValueError(f"scale_block {scale_block}, expected 1 or 16")
        shape = (n_pages, n_kv_heads, PAGE_SIZE, head_dim)
        if fmt == "bf16":
            return cls(*(torch.zeros(shape, dtype=torch.bfloat16, device=device) for _ in range(2)))
        return cls(*(torch.zeros(shape, dtype=torch.uint8, device=device) for _ in range(2)),
                   *(torch.zeros((n_pages, n_kv_heads, PAGE_SIZE // scale_block), dtype=torch.uint8, device=device)
                     for _ in range(2)))


class RowBatch:
    """The rows of a call on a PagedKv (sv_row_batch in include/sv.h).

    block_table: int32 [n_seq, pages]; first: int32 [n_seq], the position of
    each sequence's first row; n_rows: rows of the call's buffers; row_start:
    int32 [n_seq + 1], or None for n_rows / n_seq rows each; max_rows: the most
    rows of a sequence, where known (only speed depends on it). The tensors
    are read when the kernels run, so a program may change their contents
    between calls (and replays of a captured graph)."""

    def __init__(self, block_table, first, n_rows: int, *, row_start=None, max_rows: int = 0):
        if getattr(block_table, "dim", lambda: 0)() != 2 or min(block_table.shape) < 1:
            raise ValueError("block_table: must be a 2-D tensor [n_seq, pages]")
        n_seq, pages = (int(x) for x in block_table.shape)
        _check_tensor(block_table, "block_table", "torch.int32", (n_seq, pages))
        _check_tensor(first, "first", "torch.int32", (n_seq,))
        _check_tensor(row_start, "row_start", "torch.int32", (n_seq + 1,))
        if not 1 <= n_rows <= 1 << 28 or (row_start is None and n_rows % n_seq):
            raise ValueError(f"n_rows {n_rows}: must be positive (at most 2^28), and a multiple of {n_seq} without "
                             "row_start")
        if not 0 <= max_rows <= _INT_MAX:
            raise ValueError(f"max_rows {max_rows}: must not be negative, nor above {_INT_MAX}")
        if first.device != block_table.device or (row_start is not None and row_start.device != first.device):
            raise ValueError("the batch's tensors lie on different devices")
        self.n_seq, self.n_rows, self.device = n_seq, int(n_rows), block_table.device
        self.tensors = (block_table, first, row_start)
        self._workspace = {}  # bytes by (query heads, head_dim): the sizes of a batch do not change
        self._scratch = {}    # workspaces of attend by stream (see there)
        self._lock = threading.Lock()  # held while a call that uses one of them is issued
        self._c = SvRowBatch(n_seq, int(n_rows), int(max_rows), pages, _ptr(block_table), _ptr(first),
                             _ptr(row_start))
        self._p = ctypes.byref(self._c)


def _check_rows(t, name, cache, n_rows, heads):
    """Rows of heads side by side: [n_rows, heads, head_dim] bf16 whose rows may
    lie apart (a slice of a fused projection). Returns the address and the row stride."""
    d = cache.head_dim
    if t.dtype is not cache._bf16:
        raise ValueError(f"{name}: dtype {t.dtype}, expected torch.bfloat16")
    if t.device != cache.device:
        raise ValueError(f"{name}: on {t.device}, the cache on {cache.device}")
    if t.shape != (n_rows, heads, d):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {(n_rows, heads, d)}")
    at = t.data_ptr()
    if t.is_contiguous() and at % 16 == 0:
        return at, heads * d
    row, head, one = t.stride()
    if n_rows == 1:  # a lone row's stride says nothing
        row = heads * d
    if one != 1 or (head != d and heads > 1) or row < heads * d or row % 8 or at % 16:
        raise ValueError(f"{name}: needs heads side by side in rows a multiple of 8 elements apart, 16-byte "
                         f"aligned; strides {t.stride()}")
    return at, row


def _check_call(cache, rows, status):
    if rows.device != cache.device:
        raise ValueError(f"the rows' tables lie on {rows.device}, the cache on {cache.device}")
    if status is not None:
        _check_tensor(status, "status", "torch.int32", (1,))
        if status.device != cache.device:
            raise ValueError(f"status: on {status.device}, the cache on {cache.device}")


def _launch(cache, stream, call, *args):
    """call(*args, stream handle) on the cache's device; stream None: torch's current one there."""
    dev, torch_c = cache._index, cache._torch
    # (the current stream's handle without the Stream object around it: 2 us less a call)
    handle = torch_c._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
    if torch_c._cuda_getDevice() == dev:
        rc = call(*args, handle)
    else:
        import torch
        with torch.cuda.device(dev):
            rc = call(*args, handle)
    if rc != SV_OK:
        raise SvError(rc, f"{call.__name__} rejected the arguments or a CUDA call failed")


def kv_write(cache: PagedKv, rows: RowBatch, k, v, *, status=None, stream=None):
    """sv_kv_write: put the rows' K and V (bf16 [n_rows, n_kv_heads, head_dim],
    rows may lie apart) into the cache. status: int32 [1], failure bits are
    ORed into it. stream: None for torch's current one. Asynchronous: tensors
    of another stream's than the call's must be kept until it has run."""
    n, heads = rows.n_rows, cache.n_kv_heads
    kp, ks = _check_rows(k, "k", cache, n, heads)
    vp, vs = _check_rows(v, "v", cache, n, heads)
    _check_call(cache, rows, status)
    _launch(cache, stream, _lib.sv_kv_write, cache._p, rows._p, kp, ks, vp, vs, _ptr(status))


def kv_fetch(cache: PagedKv, rows: RowBatch, k_out, v_out, *, status=None, stream=None):
    """sv_kv_fetch: K and V of the rows' positions, as bf16, into k_out, v_out
    ([n_rows, n_kv_heads, head_dim]). Asynchronous."""
    n, heads = rows.n_rows, cache.n_kv_heads
    kp, ks = _check_rows(k_out, "k_out", cache, n, heads)
    vp, vs = _check_rows(v_out, "v_out", cache, n, heads)
    _check_call(cache, rows, status)
    _launch(cache, stream, _lib.sv_kv_fetch, cache._p, rows._p, kp, ks, vp, vs, _ptr(status))


def attend_workspace(cache: PagedKv, rows: RowBatch, n_q_heads: int) -> int:
    """sv_attend_workspace: bytes that attend needs besides its arguments. They grow
    with the rows and with the width of the block table, to about 512 MB (4 GB
    for the widest tables); calls of more rows run in blocks."""
    key = (n_q_heads, cache.head_dim)
    need = rows._workspace.get(key)
    if need is None:
        n = ctypes.c_int64(0)
        rc = _lib.sv_attend_workspace(cache._p, rows._p, int(n_q_heads), ctypes.byref(n))
        if rc != SV_OK:
            raise SvError(rc, f"attend_workspace({n_q_heads} query heads)")
        need = rows._workspace[key] = n.value
    return need


def _own_workspace(cache, rows, need, stream):
    """The batch's workspace on the call's stream. Work on one stream runs in
    order, so its calls may share one; allocated under that stream, its memory
    goes back to that stream's pool."""
    dev = cache._index
    if cache._torch._cuda_getDevice() != dev:
        import torch
        with torch.cuda.device(dev):
            return _own_workspace(cache, rows, need, stream)
    key = cache._torch._cuda_getCurrentRawStream(dev)
    if stream is not None and stream.cuda_stream != key:
        import torch
        with torch.cuda.stream(stream):
            return _own_workspace(cache, rows, need, None)
    capturing = cache._torch._cuda_isCurrentStreamCapturing()
    ws = None if capturing else rows._scratch.get(key)
    if ws is None or ws.numel() < need:
        import torch
        ws = torch.empty(need, dtype=torch.uint8, device=cache.device)
        if not capturing:
            rows._scratch[key] = ws
    return ws


def attend(cache: PagedKv, rows: RowBatch, q, out, *, window: int = 0, sinks: int = 0, scale=None, lse=None,
           workspace=None, status=None, stream=None):
    """sv_attend: attention of the rows over the cache. q, out: bf16 [n_rows,
    n_q_heads, head_dim] (rows may lie apart); the row at position t sees p <=
    t, or with a window only p > t - window or p < sinks. scale: None for
    1 / sqrt(head_dim). lse: fp32 [n_rows, n_q_heads] for the log-sum-exp, or
    None. workspace: uint8 tensor of attend_workspace bytes; None takes one of
    the batch's own, kept for each stream (a call that is being captured into
    a graph takes a new one from the graph's memory, so that graphs share
    none). Calls with a workspace of the caller's that may run at the same
    time, or that two threads issue on one stream, need one each. Asynchronous."""
    if getattr(q, "dim", lambda: 0)() != 3:
        raise ValueError("q: must be a 3-D tensor [n_rows, n_q_heads, head_dim]")
    heads = q.shape[1]
    if heads < 1 or heads % cache.n_kv_heads:
        raise ValueError(f"q: {heads} heads, not a multiple of the cache's {cache.n_kv_heads}")
    qp, qs = _check_rows(q, "q", cache, rows.n_rows, heads)
    op, os_ = _check_rows(out, "out", cache, rows.n_rows, heads)
    _check_call(cache, rows, status)
    if not (0 <= window <= _INT_MAX and 0 <= sinks <= _INT_MAX):
        raise ValueError(f"window {window}, sinks {sinks}: must not be negative, nor above {_INT_MAX}")
    if rows.n_seq > ATTEND_MAX_SEQ:
        raise ValueError(f"{rows.n_seq} sequences, at most {ATTEND_MAX_SEQ}")
    if lse is not None:
        _check_tensor(lse, "lse", "torch.float32", (rows.n_rows, heads))
        if lse.device != cache.device:
            raise ValueError(f"lse: on {lse.device}, the cache on {cache.device}")
    need = attend_workspace(cache, rows, heads)
    if scale is None:
        scale = cache.head_dim ** -0.5

    args = (cache._p, rows._p, heads, qp, qs, op, os_, _ptr(lse), window, sinks, scale)
    if workspace is None:
        with rows._lock:  # (the call is several launches: another thread's must not come between them)
            ws = _own_workspace(cache, rows, need, stream)
            _launch(cache, stream, _lib.sv_attend, *args, ws.data_ptr(), need, _ptr(status))
        return
    _check_buf(workspace, "workspace", "torch.uint8", need, cuda=True)
    if workspace.device != cache.device:
        raise ValueError(f"workspace: on {workspace.device}, the cache on {cache.device}")
    _launch(cache, stream, _lib.sv_attend, *args, workspace.data_ptr(), workspace.numel(), _ptr(status))


def spec_generate(target: "Context", draft: "Context", pending: int, K: int, n_new: int):
    """sv_spec_generate: greedy speculative generation of at least n_new tokens
    from `pending`, drafted by `draft` and verified by `target` (both holding
    the same tokens).  Returns (tokens committed, next pending token,
    {"verify_steps", "accepted", "proposed"})."""
    out = (ctypes.c_int32 * (n_new + max(K, 1) - 1))()
    n_out, nxt = ctypes.c_int32(0), ctypes.c_int32(0)
    stats = (ctypes.c_int32 * 3)()
    target._check(_lib.sv_spec_generate(target._h, draft._h, int(pending), int(K), int(n_new), out,
                                        ctypes.byref(n_out), ctypes.byref(nxt), stats))
    return (list(out[:n_out.value]), nxt.value,
            {"verify_steps": stats[0], "accepted": stats[1], "proposed": stats[2]})


def prefill_blocks(n: int, use_tc: bool = True) -> list:
    """sv_prefill_blocks: the row blocks sv_prefill cuts n prompt tokens into
    (use_tc: the context runs the tcgen05 linears, the default)."""
    cnt = _lib.sv_prefill_blocks(int(n), 1 if use_tc else 0, None, 0)
    if cnt < 0:
        raise SvError(cnt, f"no prefill of {n} tokens")
    arr = (ctypes.c_int32 * cnt)()
    if _lib.sv_prefill_blocks(int(n), 1 if use_tc else 0, ctypes.cast(arr, _P), cnt) != cnt:
        raise SvError(SV_E_INVAL, "prefill schedule changed size")
    return list(arr)


class Context:
    """One sequence on the GPU.

    cfg: any object with the model-shape fields of sv_config (n_layers,
    hidden, n_q_heads, n_kv_heads, head_dim, ffn, vocab, rms_eps, rope_theta,
    qk_norm, act, tie_embeddings). weights: mapping (name, layer) -> CUDA
    tensor of bf16 values (layer -1 for embed / lm_head / final_norm), the
    layout of include/sv.h; the tensors must outlive the context.
    kv_delayed: commit a verify window's K/V only after acceptance (sv_config
    kv_delayed = 1) instead of writing it and zeroing the rejected rows.
    kv_format: "bf16", or "e4m3" for a cache in 8 bits (sv_config kv_format).
    window, sinks: attend only to the last `window` positions and the first
    `sinks` (0: to all).
    """

    def __init__(self, cfg, weights, *, max_k: int, max_seq: int, max_pages: int | None = None,
                 stream=None, kv_delayed: bool = False, kv_format: str = "bf16", window: int = 0, sinks: int = 0):
        if kv_format not in ("bf16", "e4m3"):
            raise ValueError(f"kv_format {kv_format!r}, expected 'bf16' or 'e4m3'")
        if max(window, sinks) > _INT_MAX:
            raise ValueError(f"window {window}, sinks {sinks}: at most {_INT_MAX}")
        self.cfg = cfg
        self.max_k, self.max_seq = max_k, max_seq
        pages = max_pages if max_pages is not None else (max_seq + PAGE_SIZE - 1) // PAGE_SIZE
        self._c = SvConfig(cfg.n_layers, cfg.hidden, cfg.n_q_heads, cfg.n_kv_heads, cfg.head_dim,
                           cfg.ffn, cfg.vocab, cfg.rms_eps, cfg.rope_theta, cfg.qk_norm, cfg.act,
                           cfg.tie_embeddings, PAGE_SIZE, pages, max_k, max_seq, int(bool(kv_delayed)),
                           SV_KV_E4M3 if kv_format == "e4m3" else SV_KV_BF16, int(window), int(sinks))
        self._weights = weights  # keep the tensors alive
        w = SvWeights()
        w.embed = _ptr(weights[("embed", -1)])
        lm = weights.get(("lm_head", -1))
        w.lm_head = _ptr(lm) if lm is not None else w.embed
        w.final_norm = _ptr(weights[("final_norm", -1)])
        self._arrays = []
        L = max(cfg.n_layers, 1)
        for k in LAYER_KEYS:
            ptrs = (ctypes.c_void_p * L)(*[_ptr(weights.get((k, l))) for l in range(cfg.n_layers)])
            self._arrays.append(ptrs)
            setattr(w, k, ctypes.cast(ptrs, _PP))
        self._w = w
        self._stream = stream
        h = _P()
        s = _P(stream.cuda_stream) if stream is not None else _P(0)
        rc = _lib.sv_create(ctypes.byref(self._c), ctypes.byref(w), s, ctypes.byref(h))
        if rc != SV_OK:
            raise SvError(rc, "sv_create rejected the configuration or failed to allocate")
        self._h = h

    # ----------------------------------------------------------- plumbing
    def close(self):
        if getattr(self, "_h", None):
            _lib.sv_destroy(self._h)
            self._h = None

    def __del__(self):
        self.close()

    def _check(self, rc):
        if rc != SV_OK:
            raise SvError(rc, _lib.sv_last_error(self._h).decode(errors="replace"))

    # ----------------------------------------------------------- the calls
    def prefill(self, tokens, logits=None) -> int:
        _check_buf(logits, "logits", "torch.float32", self.cfg.vocab, cuda=True)
        arr = _i32_array(tokens)
        nxt = ctypes.c_int32(0)
        self._check(_lib.sv_prefill(self._h, arr, len(arr), _P(_ptr(logits)), ctypes.byref(nxt)))
        return nxt.value

    def decode(self, token: int, logits=None) -> int:
        _check_buf(logits, "logits", "torch.float32", self.cfg.vocab, cuda=True)
        nxt = ctypes.c_int32(0)
        self._check(_lib.sv_decode(self._h, int(token), _P(_ptr(logits)), ctypes.byref(nxt)))
        return nxt.value

    def verify(self, tokens, logits=None):
        arr = _i32_array(tokens)
        _check_buf(logits, "logits", "torch.float32", len(arr) * self.cfg.vocab, cuda=True)
        n = ctypes.c_int32(0)
        c = ctypes.c_int32(0)
        self._check(_lib.sv_verify(self._h, arr, len(arr), _P(_ptr(logits)), ctypes.byref(n),
                                   ctypes.byref(c)))
        return n.value, c.value

    def verify_async(self, tokens_dev, K: int, result_dev, logits=None):
        _check_buf(tokens_dev, "tokens_dev", "torch.int32", int(K))
        _check_buf(result_dev, "result_dev", "torch.int32", 4)
        _check_buf(logits, "logits", "torch.float32", int(K) * self.cfg.vocab, cuda=True)
        self._check(_lib.sv_verify_async(self._h, _P(_ptr(tokens_dev)), int(K), _P(_ptr(logits)),
                                         _P(_ptr(result_dev))))

    def reserve(self, length: int):
        self._check(_lib.sv_reserve(self._h, int(length)))

    def sync(self):
        self._check(_lib.sv_sync(self._h))

    def truncate(self, new_len: int):
        self._check(_lib.sv_truncate(self._h, int(new_len)))

    def __len__(self) -> int:
        return int(_lib.sv_seq_len(self._h))

    def kv_read(self, layer: int, first: int, count: int):
        import torch
        c = self.cfg
        k = torch.empty((count, c.n_kv_heads, c.head_dim), dtype=torch.bfloat16, device="cuda")
        v = torch.empty_like(k)
        self._check(_lib.sv_kv_read(self._h, layer, first, count, _P(k.data_ptr()),
                                    _P(v.data_ptr())))
        return k, v

    def shuffle_pages(self, seed: int):
        self._check(_lib.sv_shuffle_pages(self._h, ctypes.c_uint64(seed)))

    def trace_hidden(self, buf, max_rows: int = 0):
        """Test hook: while ``buf`` (bf16 CUDA [n_layers + 1, rows, hidden]
        for steps of up to ``max_rows`` rows) is set, every step copies its
        residual stream after each layer into it; None turns it off."""
        if buf is not None:
            _check_tensor(buf, "trace", "torch.bfloat16", (self.cfg.n_layers + 1, max_rows, self.cfg.hidden))
        self._check(_lib.sv_trace_hidden(self._h, _P(_ptr(buf)), int(max_rows)))
        self._trace = buf  # keep it alive while the library may write it

    def time_linear(self, which: int, K: int, reps: int = 3):
        """(mean device us per launch, algorithmic bytes per launch) of one
        linear class, timed on the library's stream."""
        us = ctypes.c_float(0.0)
        b = ctypes.c_double(0.0)
        self._check(_lib.sv_time_linear(self._h, int(which), int(K), int(reps), ctypes.byref(us),
                                        ctypes.byref(b)))
        return float(us.value), float(b.value)

    def kernels_per_step(self, K: int, with_head: bool = True) -> int:
        return int(_lib.sv_step_kernel_count(self._h, int(K), 1 if with_head else 0))
