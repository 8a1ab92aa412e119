"""64-bit forms of the paged-cache operators, on the CPU, in plain loops over
sequences: what the tests of tests/test_gpu_paged.py compare the kernels with.

They follow the definitions in include/sv.h from the values' side (a code is
the nearest of the 127 magnitudes e4m3 has), not from the bits' side as the
kernels do."""
from __future__ import annotations

import numpy as np

PAGE = 16
NAN_BYTE = 255


def _magnitudes():
    m = [k * 2.0 ** -9 for k in range(8)]
    for e in range(1, 16):
        m += [(8 + k) * 2.0 ** (e - 10) for k in range(8)]
    return np.array(m[:127])  # the last one's place is the NaN code


MAG = _magnitudes()
VALUE = np.concatenate([MAG, [np.nan], -MAG, [np.nan]])


def codes(y):
    """Nearest e4m3 code of doubles of magnitude at most 448, ties to the even code."""
    a = np.abs(y)
    hi = np.searchsorted(MAG, a).clip(0, 126)
    lo = (hi - 1).clip(0)
    below, above = a - MAG[lo], MAG[hi] - a
    c = np.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)
    return (c + np.where(np.signbit(y), 128, 0)).astype(np.uint8)


def exp_byte(amax):
    """Exponent byte of a block of largest magnitude amax (doubles)."""
    out = np.empty(amax.shape, np.int64)
    for i, a in np.ndenumerate(amax):
        if not np.isfinite(a):
            out[i] = NAN_BYTE
            continue
        e = -100
        while a > 448.0 * 2.0 ** e:
            e += 1
        out[i] = e + 127
    return out


def scale(b):
    b = np.asarray(b, np.int64)
    return np.where(b == NAN_BYTE, np.nan, 2.0 ** (b - 127.0))


def rows_of(first, row_start, n_rows, n_seq):
    """[(sequence, row, position)] of every row of the batch."""
    if row_start is None:
        each = n_rows // n_seq
        row_start = [s * each for s in range(n_seq + 1)]
    return [(s, r, first[s] + r - row_start[s]) for s in range(n_seq)
            for r in range(row_start[s], row_start[s + 1])]


def write(code, exps, x, table, where):
    """Rows x [n, heads, d] (float64) into code/exps in place; exps None: a
    bf16 pool holding float64 values."""
    if exps is None:
        for s, r, p in where:
            if p >= 0:
                code[table[s, p // PAGE], :, p % PAGE] = x[r]
        return
    block = PAGE // exps.shape[-1]
    if block == 1:
        for s, r, p in where:
            if p < 0:
                continue
            b = exp_byte(np.abs(x[r]).max(-1))
            pg = table[s, p // PAGE]
            bad = (b == NAN_BYTE)[:, None]
            code[pg, :, p % PAGE] = np.where(bad, 0, codes(np.where(bad, 0, x[r]) / np.where(bad, 1, scale(b)[:, None])))
            exps[pg, :, p % PAGE] = b
        return
    pages = {}
    for s, r, p in where:
        if p >= 0:
            pages.setdefault((s, p // PAGE), []).append((r, p % PAGE))
    for (s, lp), rs in pages.items():
        pg, lead = table[s, lp], min(sl for _, sl in rs)
        for h in range(code.shape[1]):
            new = exp_byte(np.array([max(np.abs(x[r, h]).max() if np.isfinite(x[r, h]).all() else np.inf for r, _ in rs)]))[0]
            old = int(exps[pg, h, 0]) if lead > 0 else 0
            b = max(int(new), old)
            for sl in range(lead):
                if b == NAN_BYTE and b != old:
                    code[pg, h, sl] = 0
                elif b != old:
                    code[pg, h, sl] = codes(VALUE[code[pg, h, sl]] * 2.0 ** (old - b))
            for r, sl in rs:
                code[pg, h, sl] = 0 if b == NAN_BYTE else codes(x[r, h] / scale(b))
            exps[pg, h, 0] = b


def read(code, exps, page, slot):
    """float64 values [heads, d] of one position."""
    if exps is None:
        return code[page, :, slot]
    block = PAGE // exps.shape[-1]
    b = scale(exps[page, :, slot // block].astype(np.int64))
    return VALUE[code[page, :, slot]] * b[:, None]


def attend(kv, table, where, q, window, sinks, sm_scale):
    """(out [n, heads, d], lse [n, heads], tol_out, tol_lse) in float64; kv =
    ((k, k_exp), (v, v_exp)).

    The tolerances count what a kernel with 16-bit operands, fp32 sums and a
    bf16 output may be off by:
      - a score s = scale sum_i q_i k_i in fp32, d products and additions each
        off by at most 2^-23 of the sum of magnitudes (an addition inside a
        tensor core may truncate): d 2^-23 scale sum |q k|; queries that lose
        bits in f16 are off by at most 2^-24 of the row's largest: another
        2^-24 scale max|q| sum |k|; its scaling and exponent, and 2^x of it,
        a few 2^-22 of |s| + 8;
      - a weight, off by e^delta - 1 and by the half step 2^-11 of f16 (two
        bf16 values are closer), so the sum of p v by (2^-11 + delta) sum p |v|
        and the denominator by delta;
      - over an 8-bit cache the f16 weight is p 2^ev over the row's largest
        such product A (ev: the value block's exponent); below 2^-14 f16's
        step no longer shrinks and it is off by up to half the last one, 2^-25,
        so the sum by 2^-25 A sum |code|;
      - fp32 sums over n positions: n 2^-23 of the sum of magnitudes, at most;
      - the half step 2^-8 of the bf16 output."""
    n, hq, d = q.shape
    n_kv = kv[0][0].shape[1]
    out, lse = np.zeros((n, hq, d)), np.full((n, hq), -np.inf)
    tol, tol_l = np.zeros((n, hq, d)), np.zeros((n, hq))
    dense = {}
    with np.errstate(all="ignore"):
        for s, r, t in where:
            seen = [p for p in range(t + 1) if window == 0 or p > t - window or p < sinks]
            if not seen:
                continue
            for p in seen:
                if (s, p) not in dense:
                    pg, sl = table[s, p // PAGE], p % PAGE
                    dense[s, p] = tuple(read(c, e, pg, sl) for c, e in kv)
                    if kv[1][1] is not None:
                        per = kv[1][1].shape[-1]
                        dense[s, p] += (scale(kv[1][1][pg, :, sl * per // PAGE].astype(np.int64)),)
            k = np.stack([dense[s, p][0] for p in seen], 1)  # [heads, p, d]
            v = np.stack([dense[s, p][1] for p in seen], 1)
            for h in range(hq):
                kh, vh, x = k[h * n_kv // hq], v[h * n_kv // hq], q[r, h]
                sc = sm_scale * (kh @ x)
                m = sc.max()
                w = np.exp(sc - m)
                lse[r, h] = m + np.log(w.sum())
                out[r, h] = w @ vh / w.sum()
                ak = np.abs(kh)
                delta = (abs(sm_scale) * (d * 2.0 ** -23 * (ak @ np.abs(x)) + 2.0 ** -24 * np.abs(x).max() * ak.sum(1))
                         + 4 * 2.0 ** -22 * (np.abs(sc) + 8)).max()
                sums = len(seen) * 2.0 ** -23
                mix = w @ np.abs(vh) / w.sum()
                # (the exponents of values of very uneven size enter the weights' logarithms: 2^-22 of up to 256)
                delta += 2.0 ** -14 * (kv[1][1] is not None) * 2.0 ** -2
                tol[r, h] = 2.0 ** -8 * np.abs(out[r, h]) + (2.0 ** -11 + 2 * delta + 2 * sums) * 1.01 * mix + 1e-38
                if kv[1][1] is not None:
                    f = np.array([dense[s, p][2][h * n_kv // hq] for p in seen])
                    tol[r, h] += 2.0 ** -25 * (w * f).max() / w.sum() * (np.abs(vh) / f[:, None]).sum(0)
                tol_l[r, h] = delta + sums + 2.0 ** -22 * (np.abs(lse[r, h]) + 8)
    return out, lse, tol, tol_l
