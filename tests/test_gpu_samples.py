"""Several continuations of a prompt, as a program runs them: pages handed out and
forked, rows written, attention to the shared prefix, log probabilities, beams
that go on from others, sequences that end, the pool packed. Every step is held
to a simulation that keeps each sequence's rows in lists."""
import numpy as np
import pytest

from . import paged_ref as ref
from . import pages_ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

PAGE = 16


def f64(t):
    return t.detach().double().cpu().numpy()


def dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("fmt,block", [("bf16", 1), ("e4m3", 1), ("e4m3", 16)])
@pytest.mark.parametrize("n_q,n_kv,d,prompt,wide", [(8, 2, 64, 45, 0), (14, 2, 128, 203, 12000), (8, 1, 256, 64, 14000)])
def test_beams(fmt, block, n_q, n_kv, d, prompt, wide):
    import greedy_speculative_decode_gb300 as sv
    g = torch.Generator().manual_seed(prompt)
    S, V, steps = 5, 700, 7
    width = (prompt + steps) // PAGE + 3 + wide // PAGE
    layers = [sv.PagedKv.empty(64, n_kv, d, fmt=fmt, scale_block=block) for _ in range(2)]
    both = sv.KvLayers(layers)
    pages = sv.KvPages.empty(S, width, 64)
    moves = torch.empty((S, 2), dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    head = torch.randn((V, n_q * d), generator=g).cuda() / (n_q * d) ** 0.5

    def randn(*shape):
        return torch.randn(shape, generator=g).bfloat16().cuda()

    def fork(**kw):
        sv.kv_fork(pages, moves, status=status, **{k: dev(v) for k, v in kw.items()})
        sv.kv_copy(both, moves, status=status)

    # what each sequence holds: its rows of K and V of each layer, one position each
    rows = [[] for _ in range(S)]

    def write(seqs, first, count):
        """`count` rows for each of the sequences, at their lengths."""
        batch = sv.RowBatch(pages.block_table, pages.length, S * count)
        kv = [(randn(S * count, n_kv, d), randn(S * count, n_kv, d)) for _ in layers]
        for cache, (k, v) in zip(layers, kv):
            sv.kv_write(cache, batch, k, v, status=status)
        back = [tuple(torch.empty_like(k) for _ in range(2)) for k, _ in kv]
        for cache, (k, v) in zip(layers, back):
            sv.kv_fetch(cache, batch, k, v, status=status)
        for s in seqs:
            for i in range(count):
                rows[s].append([(f64(k)[s * count + i], f64(v)[s * count + i]) for k, v in back])
        return batch

    def held_equals(which):
        """Every position of every sequence, in both layers, is what its rows say."""
        n = [len(rows[s]) for s in which]
        if not n or not max(n):
            return
        most = max(n)
        table = pages.block_table[which].contiguous()
        batch = sv.RowBatch(table, dev([0] * len(which)), most * len(which))
        for l, cache in enumerate(layers):
            k, v = (torch.zeros((most * len(which), n_kv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
            sv.kv_fetch(cache, batch, k, v)
            k, v = f64(k).reshape(len(which), most, n_kv, d), f64(v).reshape(len(which), most, n_kv, d)
            for i, s in enumerate(which):
                for t in range(n[i]):
                    if block == PAGE and t // PAGE >= prompt // PAGE:
                        # (a page that is written further may round its earlier codes again)
                        assert np.allclose(k[i, t], rows[s][t][l][0], atol=2.0 ** -3 * np.abs(k[i, t]).max() + 1e-9)
                        continue
                    assert np.array_equal(k[i, t], rows[s][t][l][0]) and np.array_equal(v[i, t], rows[s][t][l][1])

    # the prompt, in row 0
    fork(room=[prompt] + [0] * (S - 1))
    one = sv.RowBatch(pages.block_table[:1].contiguous(), dev([0]), prompt)
    kv = [(randn(prompt, n_kv, d), randn(prompt, n_kv, d)) for _ in layers]
    for cache, (k, v) in zip(layers, kv):
        sv.kv_write(cache, one, k, v, status=status)
        sv.kv_fetch(cache, one, k, v, status=status)
    rows[0] = [[(f64(k)[t], f64(v)[t]) for k, v in kv] for t in range(prompt)]
    pages.length[0] = prompt
    fork(source=[0] * S)
    rows = [list(rows[0]) for _ in range(S)]
    held_equals(list(range(S)))
    prefix = sv.SharedPrefix(dev([prompt]))
    alive = list(range(S))
    for step in range(steps):
        length = pages.length.cpu().tolist()
        assert length == [len(r) for r in rows]
        fork(room=[n + 1 if s in alive else 0 for s, n in enumerate(length)])
        # no page that will be written is another's
        last = [int(pages.block_table[s, length[s] // PAGE]) for s in alive]
        assert len(set(last)) == len(last) and all(int(pages.refs[p]) == 1 for p in last)
        first = pages.length
        if len(alive) < S:  # (sequences that have ended are padding)
            first = torch.where(dev([int(s in alive) for s in range(S)]) > 0, pages.length, -1)
        keep = pages.length.clone()
        pages.length.copy_(first)
        batch = write(alive, length, 1)
        q, out = randn(S, n_q, d), torch.empty((S, n_q, d), dtype=torch.bfloat16, device="cuda")
        lse = torch.empty((S, n_q), device="cuda")
        for cache, l in zip(layers, range(2)):
            sv.attend_shared(cache, batch, prefix, q, out, lse=lse, status=status)
            pool = (f64(cache.k), None) if fmt == "bf16" else (cache.k.cpu().numpy(), cache.k_exp.cpu().numpy())
            pool2 = (f64(cache.v), None) if fmt == "bf16" else (cache.v.cpu().numpy(), cache.v_exp.cpu().numpy())
            where = [(s, s, length[s]) for s in alive]
            o, w, tol, tol_l = ref.attend((pool, pool2), pages.block_table.cpu().numpy(), where, f64(q), 0, 0, d ** -0.5)
            assert (np.abs(f64(out)[alive] - o[alive]) <= tol[alive]).all()
            assert (np.abs(f64(lse)[alive] - w[alive]) <= tol_l[alive]).all()
            ended = [s for s in range(S) if s not in alive]
            assert (f64(out)[ended] == 0).all() and (f64(lse)[ended] == -np.inf).all()
        pages.length.copy_(keep)
        # scores, and who goes on from whom
        logits = (out.reshape(S, -1).float() @ head.T).contiguous()
        token = logits.argmax(1).int()
        logp, ent = torch.empty(S, device="cuda"), torch.empty(S, device="cuda")
        ids = torch.empty((S, 4), dtype=torch.int32, device="cuda")
        sv.logprobs(logits, token, logp, entropy=ent, top_ids=ids, status=status)
        want = pages_ref.logprobs(logits.double().cpu().numpy(), token.cpu().numpy()[:, None], 1.0, 4)
        assert np.allclose(f64(logp), want[0][:, 0], atol=1e-5) and np.allclose(f64(ent), want[2], atol=1e-4)
        assert np.array_equal(ids.cpu().numpy(), want[4]) and torch.equal(ids[:, 0], token)
        pages.length.add_(dev([int(s in alive) for s in range(S)]))
        if step == 2:  # the two best of all, three and two times
            best = sorted(alive, key=lambda s: -float(logp[s]))[:2]
            source = [best[0]] * 3 + [best[1]] * 2
            fork(source=source)
            rows = [list(rows[s]) for s in source]
        elif step == 4:  # one ends
            fork(source=[-1 if s == 1 else s for s in range(S)])
            rows[1] = []
            alive = [s for s in alive if s != 1]
        held_equals(alive)
    assert int(status.item()) == 0
    # packed, everything is still there
    moves = torch.empty((32, 2), dtype=torch.int32, device="cuda")
    sv.kv_compact(pages, moves, status=status)
    sv.kv_copy(both, moves, status=status)
    used = int((pages.refs > 0).sum())
    assert int(status.item()) == 0 and bool((pages.refs[:used] > 0).all()) and int(pages.block_table.max()) == used - 1
    held_equals(alive)
    sv.kv_fork(pages, torch.empty((S, 2), dtype=torch.int32, device="cuda"), source=dev([-1] * S))
    assert int(pages.refs.abs().sum()) == 0 and int(pages.block_table.max()) == -1


@pytest.mark.parametrize("fmt,block", [("bf16", 1), ("e4m3", 1), ("e4m3", 16)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_forks_copies_and_attention_with_no_kernel_between(fmt, block, d):
    """Each of these kernels may start before the one ahead of it has ended.  Tables, pages and
    exponents that the call before last has read change in between: the same bits as with
    the device waited for after every call."""
    import greedy_speculative_decode_gb300 as sv
    g = torch.Generator().manual_seed(3)
    S, n_q, n_kv, prefix, steps = 16, 32, 8, 256, 14
    width, n_pages = (56 << 20) // (S * n_kv * d * (2 if fmt == "bf16" else 1)) // PAGE + 1, 256
    shape = (n_pages, n_kv, PAGE, d)
    if fmt == "bf16":
        pool = [torch.randn(shape, generator=g).bfloat16() for _ in range(2)]
    else:
        codes = [torch.randint(0, 126, shape, generator=g) + 128 * torch.randint(0, 2, shape, generator=g) for _ in range(2)]
        exps = [torch.randint(112, 122, (n_pages, n_kv, PAGE // block), generator=g) for _ in range(2)]
        pool = [t.to(torch.uint8) for t in codes + exps]
    begin = [t.cuda() for t in pool]
    cache = sv.PagedKv(*[t.clone() for t in begin])
    pages = sv.KvPages.empty(S, width, n_pages)
    moves, status = torch.empty((S, 2), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    # rows of one prompt, of uneven lengths, whose last pages are partly filled
    lengths = [prefix + 5 + 7 * s for s in range(S)]
    room = dev([lengths[-1] + 9] * S)
    sv.kv_fork(pages, moves, source=dev([0] + [-1] * (S - 1)), room=room, status=status)
    pages.length[0] = prefix
    sv.kv_fork(pages, moves, source=dev([0] * S), room=room, status=status)
    pages.length.copy_(dev(lengths))
    tables = [t.clone() for t in (pages.block_table, pages.length, pages.held, pages.refs)]
    sources = [dev([int(x) for x in torch.randint(0, S, (S,), generator=g)]) for _ in range(steps)]
    batch, share = sv.RowBatch(pages.block_table, pages.length, S), sv.SharedPrefix(dev([prefix]))
    q = [torch.randn((S, n_q, d), generator=g).bfloat16().cuda() for _ in range(steps)]
    outs = [torch.empty_like(x) for x in q]

    def restore():
        for t, b in zip(cache.tensors, begin):
            t.copy_(b)
        for t, b in zip((pages.block_table, pages.length, pages.held, pages.refs), tables):
            t.copy_(b)
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()

    def run(wait):
        for k in range(steps):
            sv.kv_fork(pages, moves, source=sources[k], room=room, status=status)
            wait()
            sv.kv_copy(cache, moves, status=status)
            wait()
            sv.attend_shared(cache, batch, share, q[k], outs[k], status=status)
            wait()

    restore()
    run(torch.cuda.synchronize)
    want = [o.clone() for o in outs]
    assert int(status.item()) == 0 and all(torch.isfinite(w).all() for w in want)
    # not all alike: the rows do change
    assert not torch.equal(pages.length, tables[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(lambda: None)
    for _ in range(5):
        restore()
        run(lambda: None)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        restore()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    assert int(status.item()) == 0
