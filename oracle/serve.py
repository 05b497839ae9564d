"""Plain numpy definitions of the serving operators: the paged 8-bit cache
(write, read, attention) and sampling.  Slow loops over sequences, pages and
rows; codes in fp32 as the definition says, everything else in fp64.  Shares no
code with the HIP library.  Test infrastructure only."""
from __future__ import annotations

import numpy as np

INT8, E4M3 = 0, 1


def e4m3_values() -> np.ndarray:
    """The 256 values, by code (NaN at 0x7F and 0xFF)."""
    v = np.empty(256)
    for c in range(256):
        sign = -1.0 if c & 128 else 1.0
        e, m = (c >> 3) & 15, c & 7
        if e == 15 and m == 7:
            v[c] = np.nan
        elif e == 0:
            v[c] = sign * m * 2.0 ** -9
        else:
            v[c] = sign * (1 + m / 8) * 2.0 ** (e - 7)
    return v


_E4M3 = e4m3_values()
_POS = _E4M3[:127]                              # 0 .. 448, ascending with the code


def decode(codes: np.ndarray, fmt: int) -> np.ndarray:
    """fp64 values of uint8 codes."""
    return codes.view(np.int8).astype(np.float64) if fmt == INT8 else _E4M3[codes]


def encode(y: np.ndarray, fmt: int) -> np.ndarray:
    """Codes (uint8) of fp32 values: nearest, ties to even, clamped."""
    y = np.asarray(y, np.float32)
    if fmt == INT8:
        return np.clip(np.rint(y), -127, 127).astype(np.int8).view(np.uint8)
    a = np.minimum(np.abs(y.astype(np.float64)), 448.0)
    hi = np.searchsorted(_POS, a, side="left").clip(0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    pick = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi).astype(np.uint8)
    return pick | np.where(np.signbit(y), 128, 0).astype(np.uint8)


def spans(lens, cu, rows):
    """(row0, n, pos0) of each sequence, cu clamped to the rows."""
    out = []
    for b in range(len(lens)):
        r0 = min(max(int(cu[b]), 0), rows)
        r1 = min(max(int(cu[b + 1]), r0), rows)
        out.append((r0, r1 - r0, max(int(lens[b]), 0) - (r1 - r0)))
    return out


def page_of(table, pages, b, pos, page_size):
    if pos < 0 or pos // page_size >= table.shape[1]:
        return -1
    p = int(table[b, pos // page_size])
    return p if 0 <= p < pages else -1


def kv_write(codes, scales, table, lens, cu, x, fmt):
    """Write rows x [rows, heads, dim] into codes [pages, heads, page, dim] and
    scales [pages, heads], in place."""
    pages, heads, page, dim = codes.shape
    r = np.float32(1) / np.float32(127 if fmt == INT8 else 448)
    big = np.finfo(np.float32).max
    x = np.nan_to_num(np.asarray(x, np.float32), nan=0.0, posinf=big, neginf=-big)
    with np.errstate(all="ignore"):
        for b, (r0, n, pos0) in enumerate(spans(lens, cu, len(x))):
            i = 0
            while i < n:
                pos = pos0 + i
                m = min(n - i, page - pos % page)
                p = page_of(table, pages, b, pos, page)
                if p >= 0:
                    lo = pos % page
                    rows = x[r0 + i:r0 + i + m]
                    for h in range(heads):
                        old = scales[p, h]
                        s = np.float32(np.abs(rows[:, h]).max() * r)
                        if lo > 0:
                            s = np.fmax(s, old)
                            if s > old:
                                v = decode(codes[p, h, :lo], fmt).astype(np.float32) * old / s
                                codes[p, h, :lo] = encode(v, fmt)
                        codes[p, h, lo:lo + m] = encode(rows[:, h] / s, fmt) if s > 0 else 0
                        scales[p, h] = s
                i += m


def kv_rows(codes, scales, table, lens, cu, rows, fmt):
    """fp32 products code * scale of each row's token [rows, heads, dim] (0
    where it does not exist; NaN where a row belongs to no sequence)."""
    pages, heads, page, dim = codes.shape
    out = np.full((rows, heads, dim), np.nan, np.float32)
    for b, (r0, n, pos0) in enumerate(spans(lens, cu, rows)):
        for i in range(n):
            p = page_of(table, pages, b, pos0 + i, page)
            if p < 0:
                out[r0 + i] = 0
            else:
                out[r0 + i] = decode(codes[p, :, (pos0 + i) % page], fmt).astype(np.float32) * scales[p][:, None]
    return out


def kv_attention(kc, ks, vc, vs, table, lens, cu, q, fmt, scale, window=0):
    """(out, lse, A, S): fp64 [rows, heads_q, dim] and [rows, heads_q]; A = sum_j
    p_j |v_j| and S = max_j scale sum |q||k_j|, for error bounds.  NaN in rows
    that belong to no sequence."""
    pages, heads, page, dim = kc.shape
    rows, hq, _ = q.shape
    g = hq // heads
    q = np.asarray(q, np.float64)
    out, A = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    lse, S = np.full((rows, hq), np.nan), np.full((rows, hq), np.nan)
    for b, (r0, n, pos0) in enumerate(spans(lens, cu, rows)):
        top = min(max(int(lens[b]), 0), table.shape[1] * page)
        ids = np.array([page_of(table, pages, b, t, page) for t in range(top)], dtype=np.int64)
        slot = np.arange(top) % page
        there = ids >= 0
        K = np.zeros((top, heads, dim))
        V = np.zeros((top, heads, dim))
        K[there] = decode(kc[ids[there], :, slot[there]], fmt) * ks[ids[there]].astype(np.float64)[:, :, None]
        V[there] = decode(vc[ids[there], :, slot[there]], fmt) * vs[ids[there]].astype(np.float64)[:, :, None]
        for i in range(n):
            pos = pos0 + i
            see = np.flatnonzero(there & (np.arange(top) <= pos) &
                                 ((np.arange(top) > pos - window) if window > 0 else True))
            for h in range(hq):
                if len(see) == 0:
                    out[r0 + i, h], A[r0 + i, h], lse[r0 + i, h], S[r0 + i, h] = 0, 0, -np.inf, 0
                    continue
                k, v, qq = K[see, h // g], V[see, h // g], q[r0 + i, h]
                s = scale * (k @ qq)
                m = s.max()
                e = np.exp(s - m)
                p = e / e.sum()
                out[r0 + i, h] = p @ v
                A[r0 + i, h] = p @ np.abs(v)
                lse[r0 + i, h] = m + np.log(e.sum())
                S[r0 + i, h] = abs(scale) * (np.abs(k) @ np.abs(qq)).max()
    return out, lse, A, S


def sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None):
    """(tokens int32, logprobs fp64, kept counts) by sorting every row."""
    l = np.asarray(logits, np.float64).copy()
    l[np.isnan(l)] = -np.inf
    l = np.minimum(l, float(np.finfo(np.float32).max))
    rows, V = l.shape
    tok, lp, kept_n = np.empty(rows, np.int32), np.empty(rows), np.empty(rows, np.int64)
    for r in range(rows):
        row, M = l[r], l[r].max()
        if M == -np.inf:
            tok[r], lp[r], kept_n[r] = -1, -np.inf, 0
            continue
        T = 1.0 if temperature is None else float(temperature[r])
        if not T > 0:
            tok[r], lp[r], kept_n[r] = int(np.argmax(row)), 0.0, 1
            continue
        with np.errstate(all="ignore"):
            x = np.where(np.isinf(row), -np.inf, (row - M) / T)
        w = np.exp(x)
        order = np.argsort(-row, kind="stable")
        ws = w[order]
        n = V
        k = 0 if top_k is None else int(top_k[r])
        if 0 < k < V:
            n = k
        cut = n
        p = 1.0 if top_p is None else float(top_p[r])
        if p < 1:
            cum = np.cumsum(ws[:n])
            reach = np.flatnonzero(cum >= p * cum[-1])
            cut = min(cut, int(reach[0]) + 1 if len(reach) else n)
        mp = 0.0 if min_p is None else float(min_p[r])
        if mp > 0:
            cut = min(cut, int((ws >= min(mp, 1.0)).sum()))
        kept = np.sort(order[:cut])
        cum = np.cumsum(w[kept])
        i = min(int((cum <= float(u[r]) * cum[-1]).sum()), len(kept) - 1)
        tok[r], lp[r], kept_n[r] = kept[i], x[kept[i]] - np.log(cum[-1]), cut
    return tok, lp, kept_n
