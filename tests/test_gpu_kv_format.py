"""Contexts with an 8-bit cache (sv_config kv_format) and with a window and
sinks, through the C-ABI: the same promises as the bf16 contexts keep.

  - every verify row is bit-identical to single-token decode, and logits and
    cache do not depend on how the cache was built or on its pages;
  - an 8-bit cache holds the nearest codes of the values a bf16 context
    caches (its first layer, which no attention precedes);
  - logits agree with a 64-bit decoder that attends to the cached values;
  - rollback, the asynchronous call and the draft-verify loop work on them.
"""
import ctypes

import numpy as np
import pytest

import inputs
from tests import gpu_helpers as gh
from tests import paged_ref as ref
from tests import torch_ref

torch = pytest.importorskip("torch")

QWEN = inputs.shrink(inputs.QWEN3_8B, n_layers=2, hidden=512, n_q_heads=8, n_kv_heads=2, ffn=704, vocab=1024)
GEMMA = inputs.shrink(inputs.GEMMA_LIKE, n_layers=2, hidden=512, n_q_heads=8, n_kv_heads=1, ffn=704, vocab=1024)
MODELS = {"tiny": inputs.TINY, "d128": QWEN, "d256": GEMMA}
FORMS = [("e4m3", 0, 0), ("e4m3", 50, 4), ("bf16", 50, 4), ("bf16", 33, 0)]


def context(cfg, dw, fmt, window, sinks, max_k=16, max_seq=512, shuffle=None, **kw):
    import greedy_speculative_decode_gb300 as sv
    ctx = sv.Context(cfg, dw, max_k=max_k, max_seq=max_seq, kv_format=fmt, window=window, sinks=sinks, **kw)
    if shuffle is not None:
        ctx.shuffle_pages(shuffle)
    return ctx


def cache_of(ctx, cfg, n):
    return [t.clone() for layer in range(cfg.n_layers) for t in ctx.kv_read(layer, 0, n)]


def same(a, b):
    return all(torch.equal(x.view(torch.int16), y.view(torch.int16)) for x, y in zip(a, b))


@pytest.mark.gpu
@pytest.mark.parametrize("model", sorted(MODELS))
@pytest.mark.parametrize("fmt,window,sinks", FORMS)
def test_verify_rows_equal_decode_and_histories_agree(model, fmt, window, sinks):
    cfg = MODELS[model]
    _, dw = gh.make(cfg)
    prompt = inputs.prefix_tokens(0, 150, cfg.vocab)
    one = context(cfg, dw, fmt, window, sinks)
    pending = None
    for tok in prompt:  # one-token commits
        pending = one.prefill([tok])
    lg = gh.logits_buf(1, cfg.vocab)
    chain, rows = [pending], []
    for _ in range(16):
        chain.append(one.decode(chain[-1], logits=lg))
        rows.append(lg[0].clone())
    kv = cache_of(one, cfg, 166)
    for K, build in ((16, [150]), (5, [32, 1, 100, 17]), (13, [149, 1])):
        ctx = context(cfg, dw, fmt, window, sinks, shuffle=K)
        at = 0
        for n in build:
            p = ctx.prefill(prompt[at:at + n])
            at += n
        assert p == chain[0]
        i = 0
        while i + K <= 16:
            # the last draft wrong: it is rejected and rolled back
            toks = chain[i:i + K - 1] + [(chain[i + K - 1] + 1) % cfg.vocab]
            out = gh.logits_buf(K, cfg.vocab)
            n, corr = ctx.verify(toks, logits=out)
            assert (n, corr) == (K - 2, chain[i + K - 1])
            for r in range(K - 1):
                assert torch.equal(out[r], rows[i + r]), (K, i, r)
            i += n + 1
        n = len(ctx)
        assert same(cache_of(ctx, cfg, n), [t[:n] for t in kv])
        end = (n + 15) // 16 * 16
        assert all((t[n:] == 0).all() for t in cache_of(ctx, cfg, end))  # rejected rows read as zeros
        ctx.truncate(100)
        assert ctx.prefill(prompt[100:]) == chain[0]
        assert same(cache_of(ctx, cfg, 150), [t[:150] for t in kv])
        ctx.close()
    one.close()


@pytest.mark.gpu
@pytest.mark.parametrize("model", sorted(MODELS))
def test_cache_holds_the_nearest_codes(model):
    cfg = MODELS[model]
    _, dw = gh.make(cfg)
    prompt = inputs.prefix_tokens(1, 70, cfg.vocab)
    a = context(cfg, dw, "bf16", 0, 0)
    b = context(cfg, dw, "e4m3", 0, 0)
    a.prefill(prompt)
    b.prefill(prompt)
    for x, y in zip(a.kv_read(0, 0, 70), b.kv_read(0, 0, 70)):
        x, y = x.double().cpu().numpy(), y.double().cpu().numpy()
        e = ref.scale(ref.exp_byte(np.abs(x).max(-1)))[..., None]
        assert np.array_equal(ref.VALUE[ref.codes(x / e)] * e, y)


def _decoder(hw, tokens, kv, window, sinks):
    """64-bit logits of the last position, attending to the cached K and V."""
    cfg, t = hw.cfg, torch_ref._t
    n, d, hq, hkv = len(tokens), cfg.head_dim, cfg.n_q_heads, cfg.n_kv_heads
    x = t(hw.get("embed"))[torch.tensor(list(tokens))]
    i = torch.arange(n)
    seen = i[None] <= i[:, None]
    if window:
        seen &= (i[None] > i[:, None] - window) | (i[None] < sinks)

    def norm(v, w):
        return v / torch.sqrt((v * v).mean(-1, keepdim=True) + cfg.rms_eps) * t(w)

    for layer in range(cfg.n_layers):
        q = (norm(x, hw.get("attn_norm", layer)) @ t(hw.get("wqkv", layer)).T)[:, :hq * d].reshape(n, hq, d)
        if cfg.qk_norm:
            q = norm(q, hw.get("q_norm", layer))
        q = torch_ref._rope(q.transpose(0, 1), cfg.rope_theta)
        k, v = (c.double().cpu().transpose(0, 1).repeat_interleave(hq // hkv, 0) for c in kv[layer])
        s = (q @ k.transpose(1, 2) / d ** 0.5).masked_fill(~seen, -float("inf"))
        x = x + (torch.softmax(s, -1) @ v).transpose(0, 1).reshape(n, hq * d) @ t(hw.get("wo", layer)).T
        gu = norm(x, hw.get("ffn_norm", layer)) @ t(hw.get("w_gate_up", layer)).T
        g, u = gu[:, :cfg.ffn], gu[:, cfg.ffn:]
        a = torch.nn.functional.silu(g) if cfg.act == 0 else torch.nn.functional.gelu(g, approximate="tanh")
        x = x + (a * u) @ t(hw.get("w_down", layer)).T
    return (norm(x, hw.get("final_norm"))[-1] @ t(hw.get("lm_head")).T).numpy()


@pytest.mark.gpu
@pytest.mark.parametrize("model", sorted(MODELS))
@pytest.mark.parametrize("fmt,window,sinks", FORMS)
def test_logits_against_a_decoder_over_the_cached_values(model, fmt, window, sinks):
    """The decoder takes K and V as the context cached them, so what is left is
    the bf16 rounding of activations that the oracle's tolerance allows for."""
    cfg = MODELS[model]
    hw, dw = gh.make(cfg)
    prompt = inputs.prefix_tokens(2, 130, cfg.vocab)
    ctx = context(cfg, dw, fmt, window, sinks)
    lg = gh.logits_buf(1, cfg.vocab)
    ctx.prefill(prompt, logits=lg)
    kv = [ctx.kv_read(layer, 0, 130) for layer in range(cfg.n_layers)]
    want = _decoder(hw, prompt, kv, window, sinks)
    assert np.abs(lg[0].double().cpu().numpy() - want).max() <= gh.TOL_LOGIT


@pytest.mark.gpu
def test_window_longer_than_the_sequence_is_no_window():
    cfg = QWEN
    _, dw = gh.make(cfg)
    prompt = inputs.prefix_tokens(3, 90, cfg.vocab)
    out = []
    for window in (91, 500):
        ctx = context(cfg, dw, "e4m3", window, 0)
        lg = gh.logits_buf(1, cfg.vocab)
        ctx.prefill(prompt, logits=lg)
        out.append(lg)
    ctx = context(cfg, dw, "e4m3", 0, 0)
    lg = gh.logits_buf(1, cfg.vocab)
    ctx.prefill(prompt, logits=lg)
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], lg)


@pytest.mark.gpu
def test_window_with_delayed_write_through():
    """kv_delayed with a window: the same bits as write-then-truncate, queued
    without a pause between steps, over windows that straddle pages."""
    cfg = QWEN
    _, dw = gh.make(cfg)
    prompt = inputs.prefix_tokens(7, 45, cfg.vocab)
    runs = []
    for delayed in (False, True):
        ctx = context(cfg, dw, "bf16", 40, 3, kv_delayed=delayed, shuffle=2)
        pending = ctx.prefill(prompt)
        out = []
        for s in range(12):
            w = [pending] + [(pending + 3 * j + s) % cfg.vocab for j in range(1, 14)]
            lg = gh.logits_buf(14, cfg.vocab)
            n, pending = ctx.verify(w, logits=lg)
            out.append((n, pending, lg))
        runs.append((out, cache_of(ctx, cfg, len(ctx))))
    for (n, p, lg), (n2, p2, lg2) in zip(runs[0][0], runs[1][0]):
        assert (n, p) == (n2, p2) and torch.equal(lg, lg2)
    assert same(runs[0][1], runs[1][1])


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,window,sinks", FORMS[:3])
def test_asynchronous_verify_and_graphs(fmt, window, sinks, monkeypatch):
    """Queued windows against the synchronous call, and against steps launched
    without graphs or programmatic dependent launch."""
    cfg = QWEN
    _, dw = gh.make(cfg)
    prompt = inputs.prefix_tokens(4, 60, cfg.vocab)
    a = context(cfg, dw, fmt, window, sinks)
    pending = a.prefill(prompt)
    toks, lgs = [], []
    for s in range(6):
        w = [pending] + [(pending + 7 * j + s) % cfg.vocab for j in range(1, 4)]
        lg = gh.logits_buf(4, cfg.vocab)
        n, pending = a.verify(w, logits=lg)
        toks.append(w)
        lgs.append((lg, n, pending))
    kv = cache_of(a, cfg, len(a))
    b = context(cfg, dw, fmt, window, sinks)
    b.prefill(prompt)
    b.reserve(200)
    res = torch.zeros((6, 4), dtype=torch.int32, device="cuda")
    td = torch.tensor(toks, dtype=torch.int32, device="cuda")
    outs = [gh.logits_buf(4, cfg.vocab) for _ in range(6)]
    torch.cuda.synchronize()
    for s in range(6):
        b.verify_async(td[s], 4, res[s], logits=outs[s])
    b.sync()
    for s, (lg, n, p) in enumerate(lgs):
        assert torch.equal(outs[s], lg) and res[s].tolist()[:2] == [n, p]
    assert same(cache_of(b, cfg, len(b)), kv)
    for name in ("SV_NO_GRAPHS", "SV_NO_PDL", "SV_NO_TC"):
        monkeypatch.setenv(name, "1")
        c = context(cfg, dw, fmt, window, sinks)
        c.prefill(prompt)
        for w, (lg, n, p) in zip(toks, lgs):
            out = gh.logits_buf(4, cfg.vocab)
            assert c.verify(w, logits=out) == (n, p) and torch.equal(out, lg), name
        monkeypatch.delenv(name)


@pytest.mark.gpu
def test_async_windows_past_the_reserved_pages_change_nothing():
    """A window that runs past the pages: the step reports it, and no page of
    the pool that the sequence does not hold is written."""
    import greedy_speculative_decode_gb300 as sv
    cfg = inputs.TINY
    _, dw = gh.make(cfg)
    ctx = context(cfg, dw, "e4m3", 0, 0, max_seq=64)
    pending = ctx.prefill(inputs.prefix_tokens(5, 30, cfg.vocab))
    before = cache_of(ctx, cfg, 30)
    res = torch.zeros(4, dtype=torch.int32, device="cuda")
    td = torch.tensor([pending, 1, 2, 3, 4, 5], dtype=torch.int32, device="cuda")
    ctx.verify_async(td, 6, res)  # positions 30 .. 35; the pages end at 32
    with pytest.raises(sv.SvError) as e:
        ctx.sync()
    assert e.value.code == sv.SV_E_CUDA and int(res[3]) & 2
    assert same(cache_of(ctx, cfg, 30), before)


@pytest.mark.gpu
def test_speculative_loop_on_8_bit_caches():
    """sv_spec_generate: the target's greedy continuation, whatever the drafter's cache."""
    import greedy_speculative_decode_gb300 as sv
    cfg = QWEN
    _, dw = gh.make(cfg)
    prompt = inputs.prefix_tokens(6, 40, cfg.vocab)
    plain = context(cfg, dw, "e4m3", 64, 4)
    chain = gh.greedy_chain_gpu(plain, prompt, 41)
    for fmt, window in (("e4m3", 64), ("bf16", 0)):
        target = context(cfg, dw, "e4m3", 64, 4)
        draft = context(cfg, dw, fmt, window, 4)
        pending = target.prefill(prompt)
        draft.prefill(prompt)
        out, nxt, stats = sv.spec_generate(target, draft, pending, 4, 40)
        assert out[:40] == chain[:40]
        if fmt == "e4m3":  # the same model and cache: every draft is accepted
            assert stats["accepted"] == stats["proposed"]


@pytest.mark.gpu
def test_kernel_count_with_an_8_bit_cache():
    _, dw = gh.make(QWEN)
    a, b = context(QWEN, dw, "bf16", 0, 0), context(QWEN, dw, "e4m3", 0, 0)
    assert b.kernels_per_step(4) == a.kernels_per_step(4) + QWEN.n_layers


@pytest.mark.parametrize("bad", [(0, 2, 0, 0), (0, -1, 0, 0), (1, 1, 0, 0), (0, 0, -1, 0), (0, 1, 16, -2)])
def test_create_refuses(bad):
    """(kv_delayed, kv_format, window, sinks): an unknown format, delayed
    write-through of an 8-bit cache, negative windows; before any device work."""
    import greedy_speculative_decode_gb300 as sv
    c = sv.SvConfig(2, 256, 4, 2, 64, 704, 1024, 1e-6, 1e4, 1, 0, 1, 16, 8, 8, 128, *bad)
    w, h = sv.SvWeights(), ctypes.c_void_p(0)
    assert sv.lib().sv_create(ctypes.byref(c), ctypes.byref(w), None, ctypes.byref(h)) == sv.SV_E_INVAL
    assert not h.value


def test_context_refuses_an_unknown_format():
    import greedy_speculative_decode_gb300 as sv
    with pytest.raises(ValueError, match="kv_format"):
        sv.Context(inputs.TINY, {}, max_k=4, max_seq=64, kv_format="int8")
