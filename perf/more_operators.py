"""Cases of the operators for several continuations of a prompt: the pages of a
cache handed out, shared, copied and packed; attention for a batch that shares a
long prefix; log probabilities of given tokens.

Pages.  Row s of the block table holds held[s] pages for its length[s] positions,
16 a page; refs counts the rows that hold a page.
  fork     row s becomes the first min(keep[s], length[source[s]]) positions of what
           row source[s] was (-1: nothing), with pages for room[s] positions.  Whole
           pages are shared.  A last page that is not full and that others hold too
           is copied, but for the lowest row where all hold it so.  New pages are the
           lowest free ones, in the order of the rows.  The moves (from, to) are then
           copied in the pools of all layers.
  compact  the k-th highest page in use moves to the k-th lowest free one while that
           is lower; the table, the counts and the pools follow.

Shared prefix.  Sequences of a group have the same pages for the group's first
positions.  The row at position t sees p <= t:
  attend   softmax(scale * q . k) v, and the log-sum-exp.

Log probabilities of logits x, with lse = ln sum exp(x):
  logprobs x[token] - lse, the entropy lse - sum p x, and the k most probable
           tokens (ties to the lowest id).
"""
import math

import torch

own = False

PAGE = 16

# Head layouts: the framework's 8B-, 0.6B- and Gemma-shaped models, the tiny one, and a group of 7.
SHAPES = {
    "8b": (32, 8, 128),
    "0.6b": (16, 8, 128),
    "gemma": (8, 1, 256),
    "tiny": (4, 2, 64),
    "g7": (28, 4, 128),
}
VOCABS = [1024, 32003, 151936, 262144]


def _pages(name, op, shape, seqs, ctx, layers, fmt="e4m3", block=1, groups=1, room=1):
    _, n_kv, d = SHAPES[shape]
    return {"name": name, "op": op, "n_kv": n_kv, "d": d, "seqs": seqs, "ctx": ctx, "layers": layers, "fmt": fmt,
            "block": block, "groups": groups, "room": room}


def _shared(name, shape, seqs, groups, rows, prefix, more, fmt="e4m3", block=1, lse=False):
    n_q, n_kv, d = SHAPES[shape]
    return {"name": name, "op": "shared", "n_q": n_q, "n_kv": n_kv, "d": d, "seqs": seqs, "groups": groups,
            "rows": rows, "prefix": prefix, "more": more, "fmt": fmt, "block": block, "lse": lse}


def _probs(name, rows, vocab, dtype, tokens=1, top=0, entropy=True):
    return {"name": name, "op": "logprobs", "rows": rows, "vocab": vocab, "dtype": dtype, "tokens": tokens,
            "top": top, "entropy": entropy}


def listed():
    """ctx: most positions of a sequence; more: most positions behind the shared prefix, before the call's rows."""
    return [
        # one prompt becomes eight samples, each with a page to go on in: pure latency
        _pages("fork 1 to 8", "fork", "8b", 8, 1003, 2, groups=1),
        # a step of beam search over 8 prompts: rows go on from other rows, their last pages are copied
        _pages("fork beams 64x4096", "fork", "8b", 64, 4096, 4, groups=8, room=4),
        # a small pool packed after sequences have ended
        _pages("compact 6x600", "compact", "tiny", 6, 600, 2, fmt="bf16"),
        # a serving pool packed, so that its upper part can be given back
        _pages("compact 64x4096", "compact", "8b", 64, 4096, 2, block=16),
        # four samples of a short prompt, one token each: the smallest attention
        _shared("shared 4x1 prefix1024", "8b", 4, 1, 1, 1024, 40),
        # a serving batch behind one system prompt
        _shared("shared 32x1 prefix8192", "8b", 32, 1, 1, 8192, 512),
        # many samples over a long document, in a bf16 cache
        _shared("shared bf16 64x1 prefix32768", "8b", 64, 1, 1, 32768, 300, fmt="bf16"),
        # verify steps of four rows for 8 prompts of 8 samples each, a group of 7 heads, one exponent a page
        _shared("shared 64x4 g7 prefix4096", "g7", 64, 8, 4, 4096, 257, block=16),
        # one kv head of 256, bf16, odd sizes, with the log-sum-exp
        _shared("shared bf16 13x2 d256", "gemma", 13, 1, 2, 9001, 77, fmt="bf16", lse=True),
        # the token of one decode step, its entropy and 20 alternatives, from the step's fp32 logits
        _probs("logprobs 1x151936", 1, 151936, "float32", top=20),
        # a verify step's rows with the draft's and the target's token each
        _probs("logprobs 24x262144", 24, 262144, "bfloat16", tokens=2, top=5),
        # a prompt's tokens scored
        _probs("logprobs 2048x151936", 2048, 151936, "bfloat16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fork", "compact", "shared", "shared", "shared", "logprobs", "logprobs"])
    shape = rng.choice(sorted(SHAPES))
    fmt = rng.choice(["e4m3", "e4m3", "bf16"])
    block = 1 if fmt == "bf16" else rng.choice([1, 1, 16])
    if op == "logprobs":
        c = _probs("", _log(rng, 1, 2000), rng.choice(VOCABS + [_log(rng, 30, 200000) | 1]), rng.choice(["float32", "bfloat16"]),
                   tokens=rng.choice([1, 1, 2, 5]), top=rng.choice([0, 0, 1, 5, 20]), entropy=rng.random() < 0.7)
        # no more bytes than the largest listed case, and fewer where alternatives are asked for
        most = 600_000_000 if not c["top"] else 60_000_000
        while c["rows"] > 1 and c["rows"] * c["vocab"] * (4 if c["dtype"] == "float32" else 2) > most:
            c["rows"] //= 2
    elif op == "shared":
        groups = rng.choice([1, 1, 1, 2, 4, 8])
        c = _shared("", shape, groups * _log(rng, 1, 64), groups, rng.choice([1, 1, 1, 2, 4, 7]), _log(rng, 20, 32768),
                    _log(rng, 1, 700), fmt, block, rng.random() < 0.3)
        # no more products and no more cache than the largest listed case
        while c["seqs"] > groups and (c["seqs"] * c["rows"] * (c["prefix"] + c["more"]) * c["n_q"] * c["d"] > 8_000_000_000
                                      or c["seqs"] > 96):
            c["seqs"] = max(groups, c["seqs"] // 2 // groups * groups)
        while groups * c["prefix"] * c["n_kv"] * c["d"] > 33_000_000:
            c["prefix"] //= 2
    else:
        groups = rng.choice([1, 2, 4])
        c = _pages("", op, shape, groups * _log(rng, 1, 20), _log(rng, 10, 4000), rng.choice([1, 2, 3]), fmt, block, groups,
                   rng.choice([0, 1, 4, 17]))
        while c["seqs"] * c["ctx"] * c["n_kv"] * c["d"] * c["layers"] > 500_000_000:
            c["ctx"] //= 2
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs
def _pool(case, pages, g, dev):
    """K and V of a cache a program has in hand: finite codes, exponents of uneven magnitude."""
    n_kv, d = case["n_kv"], case["d"]
    out = {}
    for n in ("k", "v"):
        shape = (pages, n_kv, PAGE, d)
        if case["fmt"] == "bf16":
            x = torch.empty(shape, dtype=torch.bfloat16, device=dev).normal_(generator=g)
            out[n], out[n + "_exp"] = x.mul_(torch.exp2(torch.randn((pages, n_kv, PAGE, 1), generator=g, device=dev)).bfloat16()), None
            continue
        # each position's largest magnitude lies between 256 and 448, as the writer leaves it: codes 0x78 .. 0x7e;
        # the others are spread as those of normal values
        x = torch.empty(shape, dtype=torch.float16, device=dev).normal_(generator=g).mul_(100.0).clamp_(-448.0, 448.0)
        out[n] = x.to(torch.float8_e4m3fn).view(torch.uint8)
        del x
        out[n + "_exp"] = torch.randint(117, 122, (pages, n_kv, PAGE // case["block"]), generator=g, device=dev, dtype=torch.uint8)
    return out


def _views(pool):
    if pool["k_exp"] is None:
        return [pool["k"], pool["v"]]
    return [pool["k"].view(torch.float8_e4m3fn), pool["v"].view(torch.float8_e4m3fn), pool["k_exp"], pool["v_exp"]]


def _lengths(case):
    """Positions of each sequence: fixed by the case alone."""
    x = case["ctx"]
    return [max(1, x - (s * 7919 + 13 * s) % (x // 2 + 1)) for s in range(case["seqs"])]


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    s = {"case": case}
    {"fork": _prepare_pages, "compact": _prepare_pages, "shared": _prepare_shared, "logprobs": _prepare_probs}[case["op"]](case, s, g, dev)
    return s


def _prepare_pages(case, s, g, dev):
    seqs, per = case["seqs"], case["seqs"] // case["groups"]
    width = (case["ctx"] + max(case["room"], 1) + PAGE - 1) // PAGE + 1
    length = torch.tensor(_lengths(case), dtype=torch.int32, device=dev)
    held = (length + PAGE - 1) // PAGE
    if case["op"] == "fork":
        # the first row of each group is the prompt (one group: the others hold nothing yet)
        lead = torch.arange(seqs, device=dev) // per * per
        pages = int(held.sum()) + seqs * (2 + case["room"] // PAGE) + 7
        if case["groups"] == 1:
            length = torch.where(torch.arange(seqs, device=dev) == 0, length, 0)
            s["source"] = lead.to(torch.int32)
        else:
            s["source"] = (lead + torch.randint(0, per, (seqs,), generator=g, device=dev)).to(torch.int32)
        held = ((length + PAGE - 1) // PAGE).to(torch.int32)
        s["room"] = length[s["source"].long()] + case["room"]
    else:
        # sequences of three have ended, and their pages lie between the others'
        ended = torch.arange(seqs, device=dev) % 3 == 1
        pages = int(held.sum()) + 5
        length = torch.where(ended, 0, length)
    free_at = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    full = torch.tensor([(n + PAGE - 1) // PAGE for n in _lengths(case)], device=dev)
    begin = torch.cumsum(full, 0) - full
    j = torch.arange(width, device=dev)
    held = ((length + PAGE - 1) // PAGE).to(torch.int32)
    table = torch.where(j < held[:, None], free_at[(begin[:, None] + j).clamp(max=pages - 1)], -1)
    refs = torch.zeros(pages + 1, dtype=torch.int32, device=dev)
    refs.index_add_(0, table.reshape(-1).long().clamp(min=-1) % (pages + 1), torch.ones(table.numel(), dtype=torch.int32, device=dev))
    refs[pages] = 0
    s["table"], s["length"], s["held"], s["refs"] = table.contiguous(), length.contiguous(), held.contiguous(), refs[:pages].contiguous()
    s["new"] = [torch.empty_like(s[n]) for n in ("table", "length", "held", "refs")]
    s["moves"] = torch.empty((seqs if case["op"] == "fork" else pages // 2, 2), dtype=torch.int32, device=dev)
    s["layers"] = [_pool(case, pages, g, dev) for _ in range(case["layers"])]
    s["views"] = [v for p in s["layers"] for v in _views(p)]
    if own:
        import greedy_speculative_decode_gb300 as sv

        s["pages"] = sv.KvPages(s["table"], s["length"], s["held"], s["refs"])
        s["out"] = sv.KvPages(*s["new"])
        s["caches"] = sv.KvLayers([sv.PagedKv(p["k"], p["v"], p["k_exp"], p["v_exp"]) for p in s["layers"]])


def _more(case):
    """Positions of each sequence behind the prefix, before the call's rows."""
    x = case["more"]
    return [x - (s * 104729 + 13 * s) % (x // 2 + 1) for s in range(case["seqs"])]


def _prefix(case):
    """Shared positions of each group: whole pages, uneven where there are several."""
    x = case["prefix"]
    return [max(0, x - (k * 7919) % (x // 3 + 1)) // PAGE * PAGE for k in range(case["groups"])]


def _prepare_shared(case, s, g, dev):
    seqs, groups, rows, n_q, d = case["seqs"], case["groups"], case["rows"], case["n_q"], case["d"]
    per, prefix, more = seqs // groups, _prefix(case), _more(case)
    wide = [p // PAGE for p in prefix]
    tails = [(m + rows + PAGE - 1) // PAGE for m in more]
    width = max(wide[i // per] + tails[i] for i in range(seqs))
    pages = sum(wide) + sum(tails) + 3
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    # entry j of sequence i: its group's j-th page, or its own
    i = torch.arange(seqs, device=dev)
    w = torch.tensor(wide, device=dev)
    first_shared = (torch.cumsum(w, 0) - w)[i // per]
    t = torch.tensor(tails, device=dev)
    first_own = sum(wide) + torch.cumsum(t, 0) - t
    j, w = torch.arange(width, device=dev), w[i // per][:, None]
    at = torch.where(j < w, first_shared[:, None] + j, first_own[:, None] + j - w)
    s["table"] = torch.where(j < w + t[:, None], order[at.clamp(max=pages - 1)], -1).contiguous()
    s["shared"] = torch.tensor(prefix, dtype=torch.int32, device=dev)
    s["first"] = torch.tensor([prefix[q // per] + more[q] for q in range(seqs)], dtype=torch.int32, device=dev)
    s["own_wide"], s["wide"] = max(tails), max(max(wide), 1)
    s["pool"] = _pool(case, pages, g, dev)
    s["q"] = (2.0 * torch.randn((seqs * rows, n_q, d), generator=g, device=dev)).bfloat16()
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((seqs * rows, n_q), device=dev) if case["lse"] else None
    if own:
        import greedy_speculative_decode_gb300 as sv

        pool = s["pool"]
        s["cache"] = sv.PagedKv(pool["k"], pool["v"], pool["k_exp"], pool["v_exp"])
        s["rows"] = sv.RowBatch(s["table"], s["first"], seqs * rows)
        s["prefix"] = sv.SharedPrefix(s["shared"])


def _prepare_probs(case, s, g, dev):
    rows, vocab, k = case["rows"], case["vocab"], case["top"]
    dtype = getattr(torch, case["dtype"])
    x = torch.empty((rows, vocab), dtype=torch.bfloat16, device=dev).normal_(generator=g)
    # rows from nearly even to nearly certain, as decoding meets them; some with most tokens ruled out
    x.mul_((0.5 + 4.0 * torch.rand((rows, 1), generator=g, device=dev)).bfloat16())
    peak = torch.randint(0, vocab, (rows, 1), generator=g, device=dev)
    x.scatter_add_(1, peak, (20.0 * torch.rand((rows, 1), generator=g, device=dev)).bfloat16())
    few = (torch.arange(rows, device=dev) % 7 == 3)[:, None] & (torch.arange(vocab, device=dev) % 5 != 0)
    x.masked_fill_(few, -math.inf)
    s["logits"] = x.to(dtype)
    s["tokens"] = torch.randint(0, vocab, (rows, case["tokens"]), generator=g, device=dev, dtype=torch.int32)
    s["tokens"][:, :1] = torch.where(torch.rand((rows, 1), generator=g, device=dev) < 0.5, peak, s["tokens"][:, :1]).to(torch.int32)
    s["tokens"][:, -1:] -= s["tokens"][:, -1:] % 5  # (the last token is never one of those ruled out)
    s["out"] = torch.empty((rows, case["tokens"]), device=dev)
    s["entropy"] = torch.empty(rows, device=dev) if case["entropy"] else None
    s["top"] = (torch.empty((rows, k), device=dev), torch.empty((rows, k), dtype=torch.int32, device=dev)) if k else (None, None)


# ---------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if not own:
        return {"fork": _plain_fork, "compact": _plain_compact, "shared": _plain_shared, "logprobs": _plain_probs}[op](s)
    import greedy_speculative_decode_gb300 as sv

    if op == "fork":
        sv.kv_fork(s["pages"], s["moves"], source=s["source"], room=s["room"], out=s["out"])
        sv.kv_copy(s["caches"], s["moves"])
        return s["new"], s["moves"], s["views"]
    if op == "compact":
        sv.kv_compact(s["pages"], s["moves"], out=s["out"])
        sv.kv_copy(s["caches"], s["moves"])
        return s["new"], s["moves"], s["views"]
    if op == "shared":
        sv.attend_shared(s["cache"], s["rows"], s["prefix"], s["q"], s["out"], lse=s["lse"])
        return (s["out"], s["lse"]) if s["case"]["lse"] else s["out"]
    sv.logprobs(s["logits"], s["tokens"], s["out"], entropy=s["entropy"], top_values=s["top"][0], top_ids=s["top"][1])
    return _probs_of(s)


def _probs_of(s):
    got = [s["out"]]
    if s["case"]["entropy"]:
        got.append(s["entropy"])
    if s["case"]["top"]:
        got += [s["top"][0], s["top"][1]]
    return got


def _copy_pages(s):
    src, dst = s["moves"][:, 0].long(), s["moves"][:, 1].long()
    there = src >= 0
    src, dst = src[there], dst[there]
    names = ("k", "v") if s["layers"][0]["k_exp"] is None else ("k", "v", "k_exp", "v_exp")
    for pool in s["layers"]:
        for n in names:
            pool[n][dst] = pool[n][src]
    return s["new"], s["moves"], s["views"]


def _plain_fork(s):
    table, length, held, refs = (s[n].long() for n in ("table", "length", "held", "refs"))
    seqs, width, dev = table.shape[0], table.shape[1], table.device
    src = s["source"].long()
    some = src >= 0
    from_ = src.clamp(min=0)
    keep = torch.where(some, length[from_], 0)
    kept = (keep + PAGE - 1) // PAGE
    need = torch.where(some, (torch.maximum(keep, s["room"].long()) + PAGE - 1) // PAGE, 0)
    j = torch.arange(width, device=dev)
    new = torch.where(j < kept[:, None], table[from_], -1)
    count = refs.clone()
    ones = torch.ones(table.numel(), dtype=torch.long, device=dev)
    old = torch.where(j < held[:, None], table, -1).reshape(-1)
    count.index_add_(0, old.clamp(min=0), -ones * (old >= 0))
    count.index_add_(0, new.reshape(-1).clamp(min=0), ones * (new.reshape(-1) >= 0))
    # last pages that are not full: whose they are, and who gets a copy
    part = keep % PAGE > 0
    last = new.gather(1, (kept - 1).clamp(min=0)[:, None])[:, 0].clamp(min=0)
    row = torch.arange(seqs, device=dev)
    partly = torch.zeros_like(count).index_add_(0, last, part.long())
    lowest = torch.full_like(count, seqs).scatter_reduce_(0, last, torch.where(part, row, seqs), "amin")
    copy = part & (count[last] > 1) & ~((count[last] == partly[last]) & (lowest[last] == row))
    count.index_add_(0, last, -copy.long())
    begin = kept - copy.long()
    wanted = need - begin
    offset = torch.cumsum(wanted, 0) - wanted
    free = torch.nonzero(count == 0)[:, 0]
    fresh = (j >= begin[:, None]) & (j < need[:, None])
    page = free[(offset[:, None] + j - begin[:, None]).clamp(0, free.numel() - 1)]
    new = torch.where(fresh, page, new)
    count.index_add_(0, new.reshape(-1).clamp(min=0), fresh.reshape(-1).long())
    to = new.gather(1, begin.clamp(max=width - 1)[:, None])[:, 0]
    s["new"][0].copy_(new)
    s["new"][1].copy_(keep)
    s["new"][2].copy_(need)
    s["new"][3].copy_(count)
    s["moves"].copy_(torch.where(copy[:, None], torch.stack([last, to], 1), -1))
    return _copy_pages(s)


def _plain_compact(s):
    table, refs = s["table"].long(), s["refs"].long()
    pages = refs.numel()
    used = torch.nonzero(refs > 0)[:, 0].flip(0)
    free = torch.nonzero(refs == 0)[:, 0]
    n = min(used.numel(), free.numel())
    used, free = used[:n], free[:n]
    go = used > free
    src, dst = used[go], free[go]
    where = torch.arange(pages, device=table.device)
    where[src] = dst
    count = refs.clone()
    count[dst] = refs[src]
    count[src] = 0
    s["new"][0].copy_(torch.where(table >= 0, where[table.clamp(min=0)], -1))
    s["new"][1].copy_(s["length"])
    s["new"][2].copy_(s["held"])
    s["new"][3].copy_(count)
    s["moves"].fill_(-1)
    s["moves"][:src.numel()] = torch.stack([src, dst], 1).to(torch.int32)
    return _copy_pages(s)


def _dense(case, pool, n, pages):
    """fp32 values of the pages [..., w] as [..., heads, 16 w, d]."""
    x = pool[n][pages]
    if case["fmt"] == "bf16":
        x = x.float()
    else:
        e = (pool[n + "_exp"][pages].int() - 127).repeat_interleave(case["block"], -1).unsqueeze(-1)
        x = torch.ldexp(x.view(torch.float8_e4m3fn).float(), e)
    return x.transpose(1, 2).reshape(x.shape[0], case["n_kv"], -1, case["d"])


def _plain_shared(s):
    c, pool = s["case"], s["pool"]
    seqs, groups, rows, n_kv, d = c["seqs"], c["groups"], c["rows"], c["n_kv"], c["d"]
    per, heads = seqs // groups, c["n_q"] // c["n_kv"]
    dev = s["table"].device
    lead, shared = s["table"][::per, :s["wide"]].long(), s["shared"].long()
    k, v = (_dense(c, pool, n, lead.clamp(min=0)) for n in ("k", "v"))
    # a sequence's own pages: those behind the shared ones
    wide = (shared // PAGE).repeat_interleave(per)
    at = wide[:, None] + torch.arange(s["own_wide"], device=dev)
    mine = s["table"].long().gather(1, at.clamp(max=s["table"].shape[1] - 1)).clamp(min=0)
    k2, v2 = (_dense(c, pool, n, mine) for n in ("k", "v"))
    q = s["q"].float().reshape(seqs, rows, n_kv, heads, d).permute(0, 2, 3, 1, 4).reshape(seqs, n_kv, heads * rows, d)
    q = q * (1.0 / math.sqrt(d))
    # all rows of a group against its prefix at once
    qg = q.reshape(groups, per, n_kv, heads * rows, d).transpose(1, 2).reshape(groups, n_kv, -1, d)
    a = torch.matmul(qg, k.transpose(-1, -2))
    a = a.masked_fill((torch.arange(a.shape[-1], device=dev) >= shared[:, None])[:, None, None], -math.inf)
    b = torch.matmul(q, k2.transpose(-1, -2))
    t = s["first"].long()[:, None] + torch.arange(rows, device=dev)
    p = wide[:, None] * PAGE + torch.arange(b.shape[-1], device=dev)
    seen = (p[:, None] <= t[..., None])[:, None, None].expand(seqs, 1, heads, rows, p.shape[-1]).reshape(seqs, 1, heads * rows, -1)
    b = b.masked_fill(~seen, -math.inf)
    top = b.amax(-1, keepdim=True)
    if a.shape[-1]:
        by_seq = a.amax(-1).reshape(groups, n_kv, per, -1).transpose(1, 2).reshape(seqs, n_kv, -1, 1)
        top = torch.maximum(top, by_seq)
    w2 = torch.exp(b - top)
    w = torch.exp(a - top.reshape(groups, per, n_kv, -1).transpose(1, 2).reshape(groups, n_kv, -1, 1))
    o = torch.matmul(w, v).reshape(groups, n_kv, per, -1, d).transpose(1, 2).reshape(seqs, n_kv, -1, d)
    total = w.sum(-1).reshape(groups, n_kv, per, -1).transpose(1, 2).reshape(seqs, n_kv, -1, 1) + w2.sum(-1, keepdim=True)
    o = (o + torch.matmul(w2, v2)) / total
    s["out"].copy_(o.reshape(seqs, n_kv, heads, rows, d).permute(0, 3, 1, 2, 4).reshape(-1, c["n_q"], d))
    if not c["lse"]:
        return s["out"]
    lse = (top + torch.log(total)).reshape(seqs, n_kv, heads, rows).permute(0, 3, 1, 2)
    s["lse"].copy_(lse.reshape(-1, c["n_q"]))
    return s["out"], s["lse"]


def _plain_probs(s):
    c = s["case"]
    x = s["logits"].float()
    x = x - x.amax(-1, keepdim=True)
    e = torch.exp(x)
    total = e.sum(-1, keepdim=True)
    log_total = torch.log(total)
    s["out"].copy_(x.gather(1, s["tokens"].long()) - log_total)
    if c["entropy"]:
        s["entropy"].copy_((log_total - (e * x.clamp(min=-1e30)).sum(-1, keepdim=True) / total)[:, 0])
    if c["top"]:
        k = min(c["top"], c["vocab"])
        value, at = torch.sort(x, dim=-1, descending=True, stable=True)  # ties to the lowest id
        value = value[:, :k] - log_total
        s["top"][0].fill_(-math.inf)
        s["top"][1].fill_(-1)
        s["top"][0][:, :k] = value
        s["top"][1][:, :k] = torch.where(value > -math.inf, at[:, :k], -1).to(torch.int32)
    return _probs_of(s)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "logprobs":
        rows, n = case["rows"], case["rows"] * case["vocab"]
        out = 4 * rows * (2 * case["tokens"] + case["entropy"] + 2 * case["top"])
        return {"bytes": n * (4 if case["dtype"] == "float32" else 2) + out, "flops": 5 * n}
    n_kv, d = case["n_kv"], case["d"]
    cell = 2 * n_kv * (2 * d if case["fmt"] == "bf16" else d + 1.0 / case["block"])  # bytes of a position
    if op == "shared":
        seqs, per, rows = case["seqs"], case["seqs"] // case["groups"], case["rows"]
        prefix, more = _prefix(case), _more(case)
        cells = sum(prefix) + sum(m + rows for m in more)
        pairs = sum(rows * (prefix[i // per] + more[i]) + rows * (rows + 1) // 2 for i in range(seqs))
        n = seqs * rows * case["n_q"]
        return {"bytes": cells * (cell + 4.0 / PAGE) + 4 * n * d + (4 * n if case["lse"] else 0), "flops": 4 * pairs * case["n_q"] * d}
    held = [(n + PAGE - 1) // PAGE for n in _lengths(case)]
    seqs, per = case["seqs"], case["seqs"] // case["groups"]
    if op == "fork":
        if case["groups"] == 1:
            kept, copies = held[0] * seqs, seqs - 1
        else:  # a row's last page is copied for all but one of its continuations: 1 - (1 - 1/n)^n of the rows go on
            kept, copies = sum(held), seqs * (1.0 - 1.0 / per) ** per
        pages = sum(held) + seqs * (2 + case["room"] // PAGE) + 7
    else:
        used = sum(h for s, h in enumerate(held) if s % 3 != 1)
        pages, kept = sum(held) + 5, used
        copies = used * (1.0 - used / pages)
    return {"bytes": 8 * (kept + pages) + 2 * copies * case["layers"] * PAGE * cell, "flops": 4 * (kept + pages)}


# ---------------------------------------------------------------- 64 bits, written on its own
def _value8(codes):
    """The number each e4m3 byte stands for, from its fields."""
    b = codes.to(torch.int64)
    exp, man = (b >> 3) & 15, b & 7
    mag = torch.where(exp > 0, (8 + man).double() * torch.exp2((exp - 10).double()), man.double() * 2.0 ** -9)
    return torch.where(b >= 128, -mag, mag)


def _exact_moves(case, s):
    """The moves, page by page in plain loops."""
    table, held, length, refs = (s[n].cpu().tolist() for n in ("table", "held", "length", "refs"))
    if case["op"] == "compact":
        used = [p for p in range(len(refs)) if refs[p] > 0][::-1]
        free = [p for p in range(len(refs)) if refs[p] == 0]
        return [(a, b) for a, b in zip(used, free) if a > b]
    source, room = s["source"].cpu().tolist(), s["room"].cpu().tolist()
    for row, n in zip(table, held):
        for p in row[:n]:
            refs[p] -= 1
    kept = [table[a][:(length[a] + PAGE - 1) // PAGE] for a in source]
    for row in kept:
        for p in row:
            refs[p] += 1
    begun = {}  # page: rows that hold it as a last page that is not full
    for i, a in enumerate(source):
        if length[a] % PAGE:
            begun.setdefault(kept[i][-1], []).append(i)
    copied = [i for p, rows in begun.items() for i in (rows[1:] if refs[p] == len(rows) else rows if refs[p] > 1 else [])]
    for i in copied:
        refs[kept[i][-1]] -= 1
    free, moves = iter([p for p in range(len(refs)) if refs[p] == 0]), []
    for i, a in enumerate(source):
        if i in copied:
            moves.append((kept[i][-1], next(free)))
        for _ in range((max(length[a], room[i]) + PAGE - 1) // PAGE - len(kept[i])):
            next(free)
    return moves


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("fork", "compact"):
        moves = _exact_moves(case, s)
        for pool in s["layers"]:
            for name in ("k", "v"):
                for at in range(0, len(moves), 256):
                    some = torch.tensor(moves[at:at + 256], device="cuda")
                    pool[name][some[:, 1]] = pool[name][some[:, 0]]
        # counts, tables and exponent bytes are whole numbers, which have no error
        if case["fmt"] == "bf16":
            pools = [pool[n].double() for pool in s["layers"] for n in ("k", "v")]
        else:
            pools = [x for pool in s["layers"] for x in (_value8(pool["k"]), _value8(pool["v"]), None, None)]
        return [None] * 4, None, pools
    if case["op"] == "logprobs":
        out, entropies, tops = [], [], []
        for r in range(0, case["rows"], 64):
            x = s["logits"][r:r + 64].double()
            lse = torch.logsumexp(x, -1, keepdim=True)
            logp = x - lse
            out.append(torch.gather(logp, 1, s["tokens"][r:r + 64].long()))
            p = torch.exp(logp)
            entropies.append(-torch.where(p > 0, p * logp, 0.0).sum(-1))
            if case["top"]:
                best = torch.topk(logp, min(case["top"], case["vocab"]), dim=-1).values
                tops.append(torch.nn.functional.pad(best, (0, case["top"] - best.shape[1]), value=-math.inf))
        got = [torch.cat(out)]
        if case["entropy"]:
            got.append(torch.cat(entropies))
        if case["top"]:
            got += [torch.cat(tops), None]
        return got
    pool, prefix, more, rows = s["pool"], _prefix(case), _more(case), case["rows"]
    n_kv, per = case["n_kv"], case["seqs"] // case["groups"]
    got, logs = [], []
    for i in range(case["seqs"]):
        end = prefix[i // per] + more[i] + rows
        p = torch.arange(end, device="cuda")
        pages, slot = s["table"][i].long()[p // PAGE], p % PAGE
        kv = []
        for n in ("k", "v"):
            x = pool[n][pages, :, slot]
            kv.append(x.double() if case["fmt"] == "bf16"
                      else _value8(x) * torch.exp2(pool[n + "_exp"][pages, :, slot // case["block"]].double() - 127)[..., None])
        q = s["q"][i * rows:(i + 1) * rows].double()
        ok = p <= torch.arange(end - rows, end, device="cuda")[:, None]
        heads = []
        for h in range(n_kv):
            x = q.unflatten(1, (n_kv, -1))[:, h].transpose(0, 1)  # [heads of the group, rows, d]
            score = (x @ kv[0][:, h].T) / math.sqrt(case["d"])
            score = torch.where(ok, score, -math.inf)
            lse = torch.logsumexp(score, -1)
            heads.append((torch.exp(score - lse[..., None]) @ kv[1][:, h], lse))
        got.append(torch.cat([o for o, _ in heads]).transpose(0, 1))
        logs.append(torch.cat([x for _, x in heads]).T)
    o = torch.cat(got)
    return (o, torch.cat(logs)) if case["lse"] else o
