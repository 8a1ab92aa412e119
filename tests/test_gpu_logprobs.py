"""logprobs against the 64-bit form of pages_ref.py.

Tolerances.  With y = scale x (an fp32 constant scale log2(e), off by 2^-23 of
itself: once rounded in scale, once in the product), z = y - m is one fused
operation, off by 2^-23 |z| for the constant and half a step of the result, 2^-24
|z|; the reference m by 2^-24 |m|, the same for a whole row, so that it cancels
from every log probability but the lse itself.  2^z is off by 2^-22 and by ln2
times z's error.  With w the weights, an error of e_i = 2^-22 + 2^-22 |z_i| of each
gives
  delta = sum w_i e_i / sum w_i = 2^-22 (1 + sum p |z|)
of the sum, and adding n values along chains of at most c additions (a thread's
share, then a tree) another c 2^-24, c = 8 ceil(vocab / 4096) + 64.  In log2 units
log2 of the sum is off by 1.45 (delta + c 2^-24) and its own 2^-23 (|log2 l| + 1).  A log
probability adds 2^-22 |y - m| + 2^-23 of itself; the entropy the error of sum p z:
2 delta-like terms with |z|."""
import numpy as np
import pytest

from . import pages_ref as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def _sv():
    import greedy_speculative_decode_gb300 as sv
    return sv


def tolerances(x, scale, tokens):
    y = x * np.float64(np.float32(scale)) * np.log2(np.e)
    n, vocab = x.shape
    c = 8 * -(-vocab // 4096) + 64
    tol_l, tol_e, tol_t = np.zeros(n), np.zeros(n), np.zeros(tokens.shape)
    zs = []
    with np.errstate(all="ignore"):
        for r in range(n):
            z = np.maximum(y[r] - y[r].max(), -1000)
            w = np.exp2(z)
            p = w / w.sum()
            az = np.abs(z)
            delta = 2.0 ** -22 * (1 + (p * az).sum()) + c * 2.0 ** -24
            l2 = np.log2(w.sum())
            err = 1.45 * delta + 2.0 ** -23 * (abs(l2) + 1)
            tol_l[r] = err + 2.0 ** -22 * np.abs(y[r].max()) + 2.0 ** -23 * abs(y[r].max() + l2)
            tol_e[r] = err + 2 * (p * az * (2.0 ** -22 * (2 + az))).sum() + 2 * c * 2.0 ** -24 * (p * az).sum() + delta * (p * az).sum()
            zs.append((err, y[r].max()))
            for i, t in enumerate(tokens[r]):
                if 0 <= t < vocab and np.isfinite(y[r, t]):
                    d = abs(y[r, t] - y[r].max())
                    tol_t[r, i] = err + 2.0 ** -22 * d + 2.0 ** -22 * (d + abs(l2))
    return tol_t, tol_l, tol_e, zs


def run(x, tokens, scale=1.0, top=0, stream=None):
    sv = _sv()
    n = x.shape[0]
    out = torch.full(tokens.shape, 7.0, device="cuda")
    lse, ent = (torch.full((n,), 7.0, device="cuda") for _ in range(2))
    tv = torch.full((n, top), 7.0, device="cuda") if top else None
    ti = torch.full((n, top), 7, dtype=torch.int32, device="cuda") if top else None
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    sv.logprobs(x, tokens, out, scale=scale, lse=lse, entropy=ent, top_values=tv, top_ids=ti, status=st, stream=stream)
    torch.cuda.synchronize()
    return out, lse, ent, tv, ti, int(st.item())


def check(x, tokens, scale=1.0, top=0):
    out, lse, ent, tv, ti, st = run(x, tokens, scale, top)
    xn, tn = x.double().cpu().numpy(), tokens.cpu().numpy()
    if tn.ndim == 1:
        tn = tn[:, None]
    o, l, e, v, i = ref.logprobs(xn, tn, scale, top)
    tt, tl, te, zs = tolerances(xn, scale, tn)

    def near(got, want, tol):
        got = got.double().cpu().numpy().reshape(want.shape)
        fine = np.isfinite(want)
        assert np.array_equal(np.isnan(got), np.isnan(want))
        assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)])
        over = np.abs(got[fine] - want[fine]) - np.broadcast_to(tol, want.shape)[fine]
        assert not over.size or over.max() <= 0, over.max()

    near(out, o, tt)
    near(lse, l, tl)
    near(ent, e, te)
    if top:
        assert np.array_equal(ti.cpu().numpy(), i)
        err = np.array([z[0] for z in zs])[:, None]
        near(tv, v, err + 2.0 ** -21 * (np.abs(np.where(np.isfinite(v), v, 0)) * 1.45 + 1 + np.abs(np.where(np.isfinite(l), l, 0))[:, None]))
    assert st == (4 if ((tn < -1) | (tn >= xn.shape[1])).any() else 0)


def logits(seed, n, vocab, dtype, spread=3.0, stride=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.full((n, stride or vocab), 3.0e38, device="cuda").to(dtype)
    x = buf[:, :vocab]
    x.copy_((spread * torch.randn((n, vocab), generator=g, device="cuda")).bfloat16())  # (ties, as a model's bf16 logits have)
    return x


DTYPES = [torch.float32, torch.bfloat16]


@pytest.mark.parametrize("dtype", DTYPES, ids=["fp32", "bf16"])
@pytest.mark.parametrize("n,vocab", [(1, 1), (3, 2), (1, 31), (5, 129), (2, 1024), (1, 4097), (3, 32003), (1, 151936),
                                     (40, 9001), (2, 262144), (700, 513), (1, 600001)])
def test_logprobs(dtype, n, vocab):
    x = logits(n + vocab, n, vocab, dtype)
    g = torch.Generator(device="cuda").manual_seed(1)
    tokens = torch.randint(0, vocab, (n, 3), generator=g, device="cuda", dtype=torch.int32)
    for top in (0, 1, 20, 32):
        check(x, tokens, top=top)
    check(x, tokens[:, 0].contiguous(), scale=0.37, top=5)


@pytest.mark.parametrize("dtype", DTYPES, ids=["fp32", "bf16"])
@pytest.mark.parametrize("stride,begin", [(1001, 0), (1007, 3), (1024, 1), (1000, 5)])
def test_rows_of_any_alignment(dtype, stride, begin):
    """Odd strides and beginnings: no row lies on a boundary, and what lies beside a row has no effect."""
    n, vocab = 9, 997
    buf = logits(3, n, stride, dtype)
    buf[:, begin + vocab:] = 1.0e30
    buf[:, :begin] = 1.0e30
    x = buf.reshape(-1)[begin:].as_strided((n - 1, vocab), (stride, 1))
    tokens = torch.arange(n - 1, dtype=torch.int32, device="cuda") * 100
    if begin + vocab > stride:
        buf.clamp_(max=9.0)
    check(x, tokens, top=7)


@pytest.mark.parametrize("dtype", DTYPES, ids=["fp32", "bf16"])
def test_rows_without_a_distribution_and_impossible_tokens(dtype):
    vocab = 5000
    x = logits(5, 9, vocab, dtype)
    inf, nan = float("inf"), float("nan")
    x[0] = -inf
    x[1, 77] = inf
    x[2, 4999] = nan
    x[3, :] = -inf
    x[3, 123] = -2.5  # certain
    x[4, 5:] = -inf  # fewer possible tokens than alternatives
    x[5, ::2] = -inf
    x[6] = nan
    x[7, :] = 0.0  # all alike: ties to the lowest id
    tokens = torch.tensor([[0, -1], [77, 3], [1, 2], [123, 4], [4, 5], [1, 2], [0, 0], [4999, -1], [-2, vocab]],
                          dtype=torch.int32, device="cuda")
    for top in (1, 8, 32):
        check(x, tokens, top=top)


@pytest.mark.parametrize("dtype", DTYPES, ids=["fp32", "bf16"])
@pytest.mark.parametrize("kind", ["rising", "falling", "steps", "alike", "few", "last"])
@pytest.mark.parametrize("n", [1, 400])
def test_alternatives_of_rows_in_an_unkind_order(dtype, kind, n):
    """Values in order (every chunk's largest above all before it), long runs of
    equal ones, and all large ones in one chunk."""
    vocab = 40001
    i = torch.arange(vocab, device="cuda").float()
    row = {"rising": i / 4096, "falling": -i / 4096, "steps": torch.floor(i / 1000) * 0.25, "alike": 0 * i + 1.5,
           "few": torch.where(i % 997 == 5, 3.0, -1.0), "last": torch.where(i >= vocab - 64, 2.0 + (i % 7), 0.0)}[kind]
    x = row.to(dtype).expand(n, vocab).contiguous()
    if n > 1:
        x[1:] = x[:1] + 0.0
        x = x[:3] if vocab * n > 1 << 22 else x
        x = x.repeat(140, 1)[:400]
    tokens = torch.full((x.shape[0],), vocab - 1, dtype=torch.int32, device="cuda")
    out, lse, ent, tv, ti, _ = run(x, tokens, top=32)
    check(x[:1].contiguous(), tokens[:1], top=32)
    one = run(x[:1].contiguous(), tokens[:1], top=32)
    assert (ti == one[4]).all()  # ids do not depend on the rows beside (cut into more CTAs or fewer)


@pytest.mark.parametrize("dtype", DTYPES, ids=["fp32", "bf16"])
@pytest.mark.parametrize("vocab", [700, 5001, 151936])
@pytest.mark.parametrize("scale", [1.0, 0.5])
def test_masks_of_the_lowest_value(dtype, vocab, scale):
    # the largest finite x of row 4 is itself below what x log2(e) leaves of fp32's range
    low = torch.finfo(dtype).min
    x = torch.full((5, vocab), low, dtype=dtype, device="cuda")
    x[1, ::3] = -float("inf")
    x[2, vocab // 2] = 1.5
    x[3, 5:] = logits(9, 1, vocab - 5, dtype)[0]
    x[4, 7], x[4, 300] = low * 0.75, low * 0.75
    tokens = torch.tensor([[0, vocab - 1], [1, 3], [vocab // 2, 4], [4, 5], [7, 8]], dtype=torch.int32, device="cuda")
    for top in (0, 4, 32):
        check(x, tokens, scale=scale, top=top)
    # scale x below fp32's range
    out, lse, ent, tv, ti, st = run(x, tokens, 2.0, 4)
    most = torch.finfo(torch.float32).min
    assert out[2, 1] == most and out[3, 0] == most and lse[0] == most and lse[1] == most
    assert abs(out[0, 0].item() + np.log(vocab)) < 1e-4 and abs(ent[0].item() - np.log(vocab)) < 1e-3
    assert ti[0].tolist() == [0, 1, 2, 3] and ti[4, :2].tolist() == [7, 300] and st == 0


@pytest.mark.parametrize("dtype", DTYPES, ids=["fp32", "bf16"])
@pytest.mark.parametrize("vocab", [700, 151936])
def test_rows_far_from_zero(dtype, vocab):
    # differences beside logits that have few bits left for them
    bases = (-1.0e5, 1.0e8, -1.0e9, -1.0e10, 3.0e10, -1.0e30, 1.7e38, -2.2e38)
    x = torch.stack([torch.full((vocab,), b, dtype=dtype, device="cuda") for b in bases])
    x[:, 5:9] *= 1.0 + 2.0 * torch.finfo(dtype).eps
    x[:, 600] = -float("inf")
    tokens = torch.tensor([[5, 0, 600, vocab - 1]] * len(bases), dtype=torch.int32, device="cuda")
    for top in (0, 8):
        check(x, tokens, top=top)
    x[3, 9], x[4, 9], x[5, 9] = float("nan"), float("inf"), 2.0
    check(x, tokens, top=8)
    # the same as masks: most of a row, and what stands before and behind the rest
    x[:, 300:420] = logits(3, 8, 120, dtype)
    x[3, 9], x[4, 9] = bases[3], bases[3]
    tokens[:, 1] = 333
    check(x, tokens, top=8)


def test_large_and_far_apart_logits():
    x = torch.zeros((4, 3000), device="cuda")
    x[0] = torch.linspace(-1.0e4, 1.0e4, 3000)
    x[1, 5], x[1, 6] = 2.0 ** 100, -2.0 ** 100
    x[2] = -3.0e4
    x[3, 100] = 60.0
    tokens = torch.tensor([2999, 5, 7, 100], dtype=torch.int32, device="cuda")
    check(x, tokens, top=4)
    check(x, tokens, scale=2.0, top=4)


def test_the_same_bits_every_time_and_in_graphs_and_streams():
    sv = _sv()
    x = logits(9, 6, 151936, torch.bfloat16)
    tokens = torch.randint(0, 151936, (6,), device="cuda", dtype=torch.int32)
    a = run(x, tokens, top=20)
    for _ in range(20):
        b = run(x, tokens, top=20)
        assert all(torch.equal(p, q) for p, q in zip(a[:5], b[:5]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = run(x, tokens, top=20, stream=side)
    assert all(torch.equal(p, q) for p, q in zip(a[:5], b[:5]))
    out, ids = torch.empty(6, device="cuda"), torch.empty((6, 20), dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.logprobs(x, tokens, out, top_ids=ids)
    x.copy_(logits(10, 6, 151936, torch.bfloat16))
    g.replay()
    torch.cuda.synchronize()
    want = run(x, tokens, top=20)
    assert torch.equal(out, want[0]) and torch.equal(ids, want[4])


def test_a_steps_logits():
    """The rows of a verify step: its logits in, the greedy token among the alternatives."""
    import inputs
    from . import gpu_helpers as gh
    cfg = inputs.TINY
    dw = inputs.device_weights(cfg, seed=0, gain_std=0.1)
    ctx = gh.context(cfg, dw, max_k=8, max_seq=64)
    pending = ctx.prefill(inputs.prefix_tokens(0, 20, cfg.vocab))
    lg = gh.logits_buf(3, cfg.vocab)
    toks = [pending, 5, 9]
    _, corr = ctx.verify(toks, logits=lg)
    tokens = torch.tensor([5, 9, -1], dtype=torch.int32, device="cuda")
    check(lg, tokens, top=10)
    _, _, _, _, ti, _ = run(lg, tokens, top=10)
    assert torch.equal(ti[:, 0].long(), lg.argmax(1)) and corr in ti[:, 0].tolist()


@pytest.mark.parametrize("dtype", DTYPES, ids=["fp32", "bf16"])
def test_rows_beyond_2_to_31_elements(dtype):
    vocab, stride = 5000, (1 << 30) + 5
    flat = torch.empty(2 * stride + vocab, dtype=dtype, device="cuda")
    x = torch.as_strided(flat, (3, vocab), (stride, 1))
    x.copy_(logits(31, 3, vocab, dtype))
    tokens = torch.tensor([[0, 4999], [17, -1], [4998, 2]], dtype=torch.int32, device="cuda")
    check(x, tokens, top=5)


@pytest.mark.parametrize("dtype", DTYPES, ids=["fp32", "bf16"])
@pytest.mark.parametrize("vocab", [700, 151936])
@pytest.mark.parametrize("scale", [3.0, 1.0, 0.5, 0.25, 1.0e-3, 1.0e-20, 3.0e-29, 1.0e-30])
def test_logits_further_apart_than_fp32_reaches(dtype, vocab, scale):
    """3e38 and -3e38 in one row: a log probability is -scale 6e38, or the nearest finite value.

    The product with the scale's constant, rounded twice, and a difference, a product and a
    sum of the result's: at most five half steps, 5 * 2^-24 of the value; an ordinary log
    probability here is at most 1e2, off by less than 1e-4 (2048 steps of its size)."""
    x = torch.zeros((3, vocab), device="cuda")
    x[0, 5], x[0, 7], x[0, 9] = 3.0e38, -3.0e38, -float("inf")
    x[1, 5], x[1, 7], x[1, 9] = 3.0e38, -3.0e38, 3.0e38
    x[2], x[2, 7] = 3.0e38, -3.0e38
    x = x.to(dtype)
    tokens = torch.tensor([[5, 7, 8, 9]] * 3, dtype=torch.int32, device="cuda")
    sv = _sv()
    out, lse = torch.empty((3, 4), device="cuda"), torch.empty(3, device="cuda")
    tv, ti = torch.empty((3, 32), device="cuda"), torch.empty((3, 32), dtype=torch.int32, device="cuda")
    sv.logprobs(x, tokens, out, scale=scale, lse=lse, top_values=tv, top_ids=ti)
    torch.cuda.synchronize()
    most = np.float64(np.finfo(np.float32).max)
    o, l, _, v, i = ref.logprobs(x.double().cpu().numpy(), tokens.cpu().numpy(), scale, 32)
    for got, want in ((out, o), (lse, l), (tv, v)):
        got = got.double().cpu().numpy()
        want = np.where(np.isinf(want), want, np.clip(want, -most, most))
        assert np.array_equal(np.isinf(got), np.isinf(want))
        fine = np.isfinite(want)
        assert (np.abs(got[fine] - want[fine]) <= 5 * 2.0 ** -24 * np.abs(want[fine]) + 1e-4).all(), (got, want)
    assert np.array_equal(ti.cpu().numpy(), i)


@pytest.mark.parametrize("dtype", DTYPES, ids=["fp32", "bf16"])
@pytest.mark.parametrize("vocab", [700, 40001])
@pytest.mark.parametrize("scale", [1.0e-37, 1.0e-30, 2.0e-29, 5.0e-29, 1.0e-20, 1.0e-8, 3.0e8, 1.0e9, 1.0e12, 1.0e20, 1.0e30])
def test_scales_of_any_size(dtype, vocab, scale):
    """Impossible tokens, and masks, beside logits that the scale brings near one another or far
    apart; the same with an entropy asked for and without."""
    x = torch.full((6, vocab), -float("inf"), device="cuda")
    size = min(1.0 / scale, 1.0e38)
    row = logits(40, 1, vocab, torch.float32, spread=1.0)[0]
    x[0, ::2] = row[::2] * size
    x[1, ::3], x[1, 9] = -0.125, 0.0
    x[2, 5:40], x[2, 6] = -0.125, 20.0
    x[3] = torch.finfo(dtype).min
    x[3, 50:90], x[3, ::7] = -0.125 * size, -float("inf")
    x[4, 3], x[4, 4], x[4, 5] = -2.0e30, -1.0e30, -1.5e30
    x[5] = -1.0e30
    x[5, ::2] = -float("inf")
    x = x.to(dtype)
    tokens = torch.tensor([[0, 1, 6, 7]] * 6, dtype=torch.int32, device="cuda")
    # (a log probability and the lse may be beyond fp32's range: the nearest finite value)
    most = np.float64(np.finfo(np.float32).max)
    xn, tn = x.double().cpu().numpy(), tokens.cpu().numpy()
    o, l, e, v, i = ref.logprobs(xn, tn, scale, 8)
    tt, tl, te, zs = tolerances(xn, scale, tn)
    err = np.array([z[0] for z in zs])[:, None]
    tv_tol = err + 2.0 ** -21 * (np.abs(np.where(np.isfinite(v), v, 0)) * 1.45 + 1)

    def near(got, want, tol):
        got, want = got.double().cpu().numpy(), np.where(np.isinf(want), want, np.clip(want, -most, most))
        assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(np.isinf(got), np.isinf(want)), (got, want)
        fine = np.isfinite(want)
        tol = np.minimum(tol[fine], most) + 2.0 ** -22 * np.abs(want[fine])
        assert (np.abs(got[fine] - want[fine]) <= tol).all(), (got, want)

    for top in (0, 8):
        out, lse, ent, tv, ti, st = run(x, tokens, scale, top)
        assert st == 0
        near(out, o, tt)
        near(lse, l, tl)
        near(ent, e, te)
        if top:
            assert np.array_equal(ti.cpu().numpy(), i)
            near(tv, v, tv_tol)
    _sv().logprobs(x, tokens, out, scale=scale, lse=lse)
    torch.cuda.synchronize()
    near(out, o, tt)
    near(lse, l, tl)
