"""Cases of the paged K/V cache operators: writing rows into a cache, fetching
them back, and attention of rows over it.

A cache is paged: codes [pages, kv heads, 16 positions, head_dim], in bf16 or in
8 bits (e4m3).  An 8-bit cache keeps one power-of-two exponent (e8m0 byte b, the
value 2^(b - 127)) for each kv head and block of 1 or 16 positions: a block whose
largest magnitude is a takes the smallest exponent e >= -100 with a <= 448 * 2^e.

A batch is n_seq sequences, each with its pages in a row of the block table.
Sequence s brings rows(s) rows at positions first[s], first[s] + 1, ...; the
rows of all sequences lie one behind the other.

  write   rounds the rows' K and V to codes and puts them into their pages.  With
          blocks of 16 positions a block that holds earlier positions keeps or
          raises its exponent, and its codes are rounded anew when it rises.
  fetch   the reverse: K and V of the rows' positions as bf16.
  attend  softmax(scale * q . k) v over the positions a row sees: those up to its
          own, and with a window only the last `window` of them and the first
          `sinks` of the sequence.
"""
import math

import torch

own = False

PAGE = 16
EXP_MIN = -100  # smallest exponent of a block

# Head layouts: the framework's 8B-, 0.6B- and Gemma-shaped models, the tiny one, and a group of 7.
SHAPES = {
    "8b": (32, 8, 128),
    "0.6b": (16, 8, 128),
    "gemma": (8, 1, 256),
    "tiny": (4, 2, 64),
    "g7": (28, 4, 128),
}


def _case(name, op, shape, seqs, rows, ctx, fmt="e4m3", block=1, window=0, sinks=0, ragged=False, lse=False):
    n_q, n_kv, d = SHAPES[shape]
    return {"name": name, "op": op, "n_q": n_q, "n_kv": n_kv, "d": d, "seqs": seqs, "rows": rows, "ctx": ctx,
            "fmt": fmt, "block": block, "window": window, "sinks": sinks, "ragged": ragged, "lse": lse}


def listed():
    """rows: most rows of a sequence; ctx: most positions held before them."""
    return [
        # one verify step's K/V of one layer: pure latency
        _case("write verify 1x4", "write", "8b", 1, 4, 1024),
        # a long prompt's K/V, read out of the fused projection's rows
        _case("write prompt 1x8191", "write", "8b", 1, 8191, 0),
        # a batch that appends runs of uneven length to pages already begun, one exponent a page
        _case("write block16 48x61", "write", "8b", 48, 61, 1000, block=16, ragged=True),
        # a cached prefix read back, from the middle of a page, heads of 256
        _case("fetch 1x4097 d256", "fetch", "gemma", 1, 4097, 87),
        # uneven parts of many sequences, one exponent a page
        _case("fetch ragged 24x700", "fetch", "8b", 24, 700, 300, block=16, ragged=True),
        # single-token decode of one sequence: the smallest call
        _case("decode 1x1 ctx1024", "attend", "8b", 1, 1, 1024),
        # single-token decode of a serving batch with uneven contexts
        _case("decode 32x1 ctx8192", "attend", "8b", 32, 1, 8191, ragged=True),
        # a verify step of four rows over a long context
        _case("verify 1x4 ctx32768", "attend", "8b", 1, 4, 32764),
        # wide verify steps of several sequences, one exponent a page
        _case("verify 8x16 ctx4096", "attend", "8b", 8, 16, 4080, block=16, ragged=True),
        # streaming decode: a window and the first tokens over long contexts
        _case("window 16x4 ctx32768", "attend", "8b", 16, 4, 32764, window=4096, sinks=4, ragged=True),
        # a window over a bf16 cache, one kv head of 256
        _case("window bf16 4x8 d256", "attend", "gemma", 4, 8, 9001, fmt="bf16", window=1024, sinks=5, ragged=True),
        # a prefill block of 128 rows behind a cached prefix, with its log-sum-exp
        _case("prefill 1x128 ctx4096", "attend", "8b", 1, 128, 4001, lse=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "fetch", "attend", "attend", "attend"])
    n_q, n_kv, d = SHAPES[rng.choice(sorted(SHAPES))]
    c = {"op": op, "n_q": n_q, "n_kv": n_kv, "d": d, "seqs": _log(rng, 1, 48), "fmt": "e4m3", "block": rng.choice([1, 1, 16]),
         "window": 0, "sinks": 0, "ragged": rng.random() < 0.6, "lse": False}
    if op == "attend":
        c["rows"] = _log(rng, 1, 128)
        c["ctx"] = _log(rng, 1, 32768)
        c["fmt"] = rng.choice(["e4m3", "e4m3", "bf16"])
        c["lse"] = rng.random() < 0.3
        if rng.random() < 0.4:
            c["window"] = _log(rng, 1, 8192)
            c["sinks"] = rng.choice([0, 1, 4, 17])
        # no more cache, and no more products, than the largest listed case
        while c["seqs"] * (c["ctx"] + c["rows"]) * n_kv * d > 200_000_000 or c["seqs"] * c["rows"] * (c["ctx"] + c["rows"]) * n_q * d > 1_200_000_000:
            if c["seqs"] > 1:
                c["seqs"] //= 2
            else:
                c["rows"] = max(1, c["rows"] // 2)
    else:
        c["rows"] = _log(rng, 1, 8000)
        c["ctx"] = _log(rng, 1, 3000)
        while c["seqs"] * c["rows"] * n_kv * d > 8_000_000:
            if c["seqs"] > 1:
                c["seqs"] //= 2
            else:
                c["rows"] //= 2
    if c["fmt"] == "bf16":
        c["block"] = 1
    return c


def _layout(case):
    """(rows, first position) of each sequence: fixed by the case alone."""
    n, r, x = case["seqs"], case["rows"], case["ctx"]
    if not case["ragged"]:
        return [r] * n, [x] * n
    return ([max(1, r - (s * 7919) % max(1, r)) if s % 4 else r for s in range(n)],
            [x - (s * 104729 + 13 * s) % (x // 2 + 1) for s in range(n)])


def _dims(case):
    rows, first = _layout(case)
    width = max((f + r + PAGE - 1) // PAGE for f, r in zip(first, rows))
    return rows, first, width, sum(rows)


def _block_exponent(amax):
    """Smallest e >= EXP_MIN with amax <= 448 * 2^e (exact: a power of two and a comparison)."""
    m, x = torch.frexp(amax)
    e = torch.where(m <= 0.875, x - 9, x - 8)
    return torch.where(amax > 0, e, torch.full_like(e, EXP_MIN)).clamp(min=EXP_MIN)


def _pow2(e):
    return torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)


def _codes(x, e):
    """x / 2^e as e4m3 bytes; e broadcast over x."""
    return torch.ldexp(x, -e).to(torch.float8_e4m3fn).view(torch.uint8)


def _dequant(codes, exps):
    """fp32 values of codes [..., 16, d] with exponent bytes [..., 16 / block]."""
    e = exps.to(torch.int32) - 127
    e = e.repeat_interleave(PAGE // exps.shape[-1], dim=-1).unsqueeze(-1)
    return codes.view(torch.float8_e4m3fn).float() * _pow2(e)


def _fresh_cache(case, pages, g, dev):
    """K and V pools a program has in hand: rows of uneven magnitude, as heads and tokens have them."""
    n_kv, d, out = case["n_kv"], case["d"], {}
    for n in ("k", "v"):
        codes, exps = [], []
        for p0 in range(0, pages, 16384):
            p = min(16384, pages - p0)
            x = torch.randn((p, n_kv, PAGE, d), generator=g, device=dev)
            x *= torch.exp2(2.0 * torch.randn((p, n_kv, PAGE, 1), generator=g, device=dev).clamp(-3, 3) - (1 if n == "k" else 0))
            x = x.bfloat16()
            if case["fmt"] == "bf16":
                codes.append(x)
                continue
            amax = x.float().abs().amax(-1).unflatten(-1, (-1, case["block"])).amax(-1)
            e = _block_exponent(amax)
            codes.append(_codes(x.float(), e.repeat_interleave(case["block"], -1).unsqueeze(-1)))
            exps.append((e + 127).to(torch.uint8))
        out[n] = torch.cat(codes)
        out[n + "_exp"] = torch.cat(exps) if exps else None
    return out


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    rows, first, width, n = _dims(case)
    n_q, n_kv, d, seqs = case["n_q"], case["n_kv"], case["d"], case["seqs"]
    pages = seqs * width + 5
    s = {"case": case, "pool": _fresh_cache(case, pages, g, dev)}
    s["table"] = torch.randperm(pages, generator=g, device=dev)[: seqs * width].to(torch.int32).reshape(seqs, width)
    s["first"] = torch.tensor(first, dtype=torch.int32, device=dev)
    starts = [0]
    for r in rows:
        starts.append(starts[-1] + r)
    s["row_start"] = torch.tensor(starts, dtype=torch.int32, device=dev)
    s["n"], s["max_rows"] = n, max(rows)
    if case["op"] == "write":
        # rows of a fused projection: q heads, k heads, v heads side by side
        qkv = torch.randn((n, n_q + 2 * n_kv, d), generator=g, device=dev)
        qkv *= torch.exp2(1.5 * torch.randn((n, n_q + 2 * n_kv, 1), generator=g, device=dev))
        qkv = qkv.bfloat16()
        s["qkv"], s["k"], s["v"] = qkv, qkv[:, n_q:n_q + n_kv], qkv[:, n_q + n_kv:]
    elif case["op"] == "fetch":
        s["k_out"] = torch.empty((n, n_kv, d), dtype=torch.bfloat16, device=dev)
        s["v_out"] = torch.empty_like(s["k_out"])
    else:
        s["q"] = (2.0 * torch.randn((n, n_q, d), generator=g, device=dev)).bfloat16()
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((n, n_q), device=dev) if case["lse"] else None
    if own:
        import greedy_speculative_decode_gb300 as sv

        pool = s["pool"]
        s["cache"] = sv.PagedKv(pool["k"], pool["v"], pool["k_exp"], pool["v_exp"])
        s["rows"] = sv.RowBatch(s["table"], s["first"], n, row_start=s["row_start"] if case["ragged"] else None, max_rows=s["max_rows"])
    return s


def run(s):
    if own:
        import greedy_speculative_decode_gb300 as sv

        c, pool = s["case"], s["pool"]
        if c["op"] == "write":
            sv.kv_write(s["cache"], s["rows"], s["k"], s["v"])
        elif c["op"] == "fetch":
            sv.kv_fetch(s["cache"], s["rows"], s["k_out"], s["v_out"])
            return s["k_out"], s["v_out"]
        else:
            sv.attend(s["cache"], s["rows"], s["q"], s["out"], window=c["window"], sinks=c["sinks"], lse=s["lse"])
            return (s["out"], s["lse"]) if c["lse"] else s["out"]
        return _written(pool)
    return {"write": _plain_write, "fetch": _plain_fetch, "attend": _plain_attend}[s["case"]["op"]](s)


def _written(pool):
    return [pool["k"].view(torch.float8_e4m3fn), pool["v"].view(torch.float8_e4m3fn), pool["k_exp"], pool["v_exp"]]


def _places(s):
    """(sequence, position) of every row."""
    i = torch.arange(s["n"], device="cuda")
    seq = torch.searchsorted(s["row_start"][1:].long(), i, right=True)
    return seq, s["first"][seq].long() + i - s["row_start"][seq].long()


def _plain_write(s):
    c, pool = s["case"], s["pool"]
    seq, pos = _places(s)
    page, slot = s["table"][seq, pos // PAGE].long(), pos % PAGE
    for n in ("k", "v"):
        x = s[n].float()
        codes, exps = pool[n], pool[n + "_exp"]
        if c["block"] == 1:
            e = _block_exponent(x.abs().amax(-1))
            codes[page, :, slot] = _codes(x, e.unsqueeze(-1))
            exps[page, :, slot] = (e + 127).to(torch.uint8)
            continue
        # one exponent a page: the new rows' largest value of each page and head, and whether the page was begun before
        top = torch.zeros((codes.shape[0], x.shape[1]), device="cuda")
        top.index_reduce_(0, page, x.abs().amax(-1), "amax")
        begun = torch.full((codes.shape[0],), PAGE, device="cuda", dtype=torch.long)
        begun.scatter_reduce_(0, page, slot, "amin")  # first slot written
        held = torch.unique(page)
        old = exps[held, :, 0].to(torch.int32) - 127
        e = _block_exponent(top[held])
        e = torch.where(begun[held].unsqueeze(-1) > 0, torch.maximum(e, old), e)
        values = codes[held].view(torch.float8_e4m3fn).float()
        again = _codes(values, (e - old).unsqueeze(-1).unsqueeze(-1))
        earlier = torch.arange(PAGE, device="cuda") < begun[held].unsqueeze(-1)
        codes[held] = torch.where(earlier[:, None, :, None], again, codes[held])
        exps[held, :, 0] = (e + 127).to(torch.uint8)
        at = exps[page, :, 0].to(torch.int32) - 127
        codes[page, :, slot] = _codes(x, at.unsqueeze(-1))
    return _written(pool)


def _plain_fetch(s):
    c, pool = s["case"], s["pool"]
    seq, pos = _places(s)
    page, slot = s["table"][seq, pos // PAGE].long(), pos % PAGE
    for n in ("k", "v"):
        e = pool[n + "_exp"][page, :, slot // c["block"]].to(torch.int32) - 127
        s[n + "_out"].copy_(pool[n][page, :, slot].view(torch.float8_e4m3fn).float() * _pow2(e).unsqueeze(-1))
    return s["k_out"], s["v_out"]


def _plain_attend(s):
    c, pool = s["case"], s["pool"]
    n_kv, d, seqs = c["n_kv"], c["d"], c["seqs"]
    group, most = c["n_q"] // n_kv, s["max_rows"]
    dense = []
    for n in ("k", "v"):
        codes = pool[n][s["table"].long()]  # [seqs, width, heads, 16, d]
        x = codes.float() if c["fmt"] == "bf16" else _dequant(codes, pool[n + "_exp"][s["table"].long()])
        dense.append(x.permute(0, 2, 1, 3, 4).reshape(seqs, n_kv, -1, d))
    k, v = dense
    seq, pos = _places(s)
    i = pos - s["first"][seq].long()
    q = torch.zeros((seqs, most, n_kv, group, d), device="cuda")
    q[seq, i] = s["q"].float().reshape(-1, n_kv, group, d)
    q = q.permute(0, 2, 3, 1, 4).reshape(seqs, n_kv, group * most, d)
    score = torch.matmul(q, k.transpose(-1, -2)) * (1.0 / math.sqrt(d))
    t = s["first"].long()[:, None] + torch.arange(most, device="cuda")  # position of each row
    p = torch.arange(k.shape[2], device="cuda")
    seen = p <= t[..., None]
    if c["window"]:
        seen &= (p > t[..., None] - c["window"]) | (p < c["sinks"])
    seen = seen[:, None, None].expand(seqs, 1, group, most, p.numel()).reshape(seqs, 1, group * most, -1)
    score = score.masked_fill(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    w = torch.exp(score - top)
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w, v) / total
    o = o.reshape(seqs, n_kv, group, most, d).permute(0, 3, 1, 2, 4)[seq, i]
    s["out"].copy_(o.reshape(-1, c["n_q"], d))
    if not c["lse"]:
        return s["out"]
    lse = (top + torch.log(total)).reshape(seqs, n_kv, group, most).permute(0, 3, 1, 2)[seq, i]
    s["lse"].copy_(lse.reshape(-1, c["n_q"]))
    return s["out"], s["lse"]


def _seen_pairs(case):
    """(pairs of a row and a position it sees, positions that some row of their sequence sees)."""
    rows, first, _, _ = _dims(case)
    w, sinks, pairs, cells = case["window"], case["sinks"], 0, 0
    for r, f in zip(rows, first):
        if not w:
            pairs += r * f + r * (r + 1) // 2
            cells += f + r
            continue
        for t in range(f, f + r):
            lo = max(0, t - w + 1)
            pairs += t + 1 - lo + min(sinks, lo)
        lo = max(0, f - w + 1)
        cells += f + r - lo + min(sinks, lo)
    return pairs, cells


def work(case):
    rows, first, width, n = _dims(case)
    n_q, n_kv, d = case["n_q"], case["n_kv"], case["d"]
    if case["op"] == "attend":
        pairs, cells = _seen_pairs(case)
        cell = 2 * n_kv * (2 * d if case["fmt"] == "bf16" else d + 1.0 / case["block"])
        return {"bytes": cells * (cell + 4.0 / PAGE) + 4 * n * n_q * d + (4 * n * n_q if case["lse"] else 0), "flops": 4 * pairs * n_q * d}
    cell = 2 * n_kv * (2 * d + d + 1.0 / case["block"])
    return {"bytes": n * (cell + 4.0 / PAGE), "flops": 2 * n * 2 * n_kv * d}


# ---------------------------------------------------------------- 64 bits, written on its own
def _value8(codes):
    """The number each e4m3 byte stands for, from its fields."""
    b = codes.to(torch.int64)
    exp, man = (b >> 3) & 15, b & 7
    mag = torch.where(exp > 0, (8 + man).double() * torch.exp2((exp - 10).double()), man.double() * 2.0 ** -9)
    return torch.where(b >= 128, -mag, mag)


def _round8(y):
    """Doubles of magnitude at most 448 to the nearest e4m3 value, ties to even."""
    a = y.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.sign(y) * torch.round(a / step) * step


def _need(a):
    """The exponent of a block of largest magnitude a (doubles), found by comparison."""
    e = torch.full(a.shape, float(EXP_MIN), dtype=torch.float64, device=a.device)
    guess = torch.floor(torch.log2(a.clamp(min=1e-300) / 448.0)) - 1
    for k in range(4):  # the smallest of a few neighbours that is large enough
        t = guess + (3 - k)
        e = torch.where((a <= 448.0 * torch.exp2(t)) & (t >= EXP_MIN), t, e)
    return e


def exact(case, seed):
    s = prepare(case, seed)
    pool, rows, first = s["pool"], _layout(case)[0], _layout(case)[1]
    n_kv, d, b = case["n_kv"], case["d"], case["block"]
    table = s["table"].cpu()
    if case["op"] == "write":
        if max(rows) * case["seqs"] > 200_000:
            return None
        out = []
        for n in ("k", "v"):
            value, exps = _value8(pool[n]), pool[n + "_exp"].double() - 127
            at = 0
            for q in range(case["seqs"]):
                x = s[n][at:at + rows[q]].double().transpose(0, 1)  # [heads, rows, d]
                at += rows[q]
                a, z = first[q], first[q] + rows[q]
                pages = table[q, a // PAGE:(z - 1) // PAGE + 1].long().cuda()
                lead, slots = a % PAGE, len(pages) * PAGE
                pad = torch.zeros((n_kv, slots, d), dtype=torch.float64, device="cuda")
                pad[:, lead:lead + rows[q]] = x
                new = torch.zeros(slots, dtype=torch.bool, device="cuda")
                new[lead:lead + rows[q]] = True
                old_v = value[pages].transpose(0, 1).reshape(n_kv, slots, d)
                old_e = exps[pages].transpose(0, 1).reshape(n_kv, slots // b)
                e = _need(pad.abs().amax(-1).reshape(n_kv, slots // b, b).amax(-1))
                if b == PAGE and lead:
                    e[:, 0] = torch.maximum(e[:, 0], old_e[:, 0])
                touched = new.reshape(-1, b).any(-1)
                e = torch.where(touched, e, old_e)
                full = e.repeat_interleave(b, -1).unsqueeze(-1)
                was = old_e.repeat_interleave(b, -1).unsqueeze(-1)
                fresh = _round8(pad / torch.exp2(full))
                before = torch.arange(slots, device="cuda") < lead
                kept = torch.where(before[:, None] & (full != was), _round8(old_v * torch.exp2(was - full)), old_v)
                got = torch.where(new[:, None], fresh, kept)
                value[pages] = got.reshape(n_kv, len(pages), PAGE, d).transpose(0, 1)
                exps[pages] = e.reshape(n_kv, len(pages), PAGE // b).transpose(0, 1)
            out.append((value, exps))
        # the exponent bytes are whole numbers, which have no error
        return [out[0][0], out[1][0], None, None]
    got, lses, at = [[], []], [], 0
    for q in range(case["seqs"]):
        a, z = first[q], first[q] + rows[q]
        if case["op"] == "attend":
            lo = max(0, a - case["window"] + 1) if case["window"] else 0
            p = torch.arange(z)
            p = p[(p >= lo) | (p < case["sinks"])].cuda()
        else:
            p = torch.arange(a, z).cuda()
        pages, slot = s["table"][q].long()[p // PAGE], p % PAGE
        kv = []
        for n in ("k", "v"):
            if case["fmt"] == "bf16":
                kv.append(pool[n][pages, :, slot].double())
            else:
                kv.append(_value8(pool[n][pages, :, slot]) * torch.exp2(pool[n + "_exp"][pages, :, slot // b].double() - 127)[..., None])
        if case["op"] == "fetch":
            got[0].append(kv[0])
            got[1].append(kv[1])
            continue
        x = s["q"][at:at + rows[q]].double()
        at += rows[q]
        t = torch.arange(a, z).cuda()[:, None]
        ok = p[None] <= t
        if case["window"]:
            ok = ok & ((t - p[None] < case["window"]) | (p[None] < case["sinks"]))
        heads, logs = [], []
        for h in range(case["n_q"]):
            k, v = (y[:, h // (case["n_q"] // n_kv)] for y in kv)
            score = (x[:, h] @ k.T) / math.sqrt(d)
            score[~ok] = -math.inf
            logs.append(torch.logsumexp(score, -1))
            heads.append(torch.exp(score - logs[-1][:, None]) @ v)
        got[0].append(torch.stack(heads, 1))
        lses.append(torch.stack(logs, 1))
    if case["op"] == "fetch":
        return torch.cat(got[0]), torch.cat(got[1])
    o = torch.cat(got[0])
    return (o, torch.cat(lses)) if case["lse"] else o
