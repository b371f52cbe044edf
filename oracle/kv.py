"""The 8-bit key/value cache: block tables from lengths, the append that
quantizes into pages (E4M3 elements, one E8M0 scale per page and head), and
causal attention over the pages.

Layouts: k_codes [N, H, P, D], v_codes [N, H, D, P] (uint8 E4M3), scales
[N, H] (uint8 E8M0).  The scale of a block is the least power of two 2^(c-127)
with amax <= 448 * 2^(c-127) (c clamped at 0); it only grows while a page
fills, and the codes already there follow it.  Derived from the formats alone:
parity unpinned.
"""
from __future__ import annotations

import numpy as np

from .e4m3 import e4m3_from_f32
from .formats import e4m3_decode, e8m0_decode


def blocks(ctx_lens, new_lens, free_pages, cursor, page, table, tokens):
    """One step's tables.  Returns (table, slots, positions, cu_new, kv_lens, state)."""
    table = np.array(table, dtype=np.int64)
    slots = np.full(tokens, -1, np.int64)
    positions = np.full(tokens, -1, np.int64)
    cu, kv = [0], []
    at, used, refused, row = max(int(cursor), 0), max(int(cursor), 0), 0, 0
    for i, (c, n) in enumerate(zip(ctx_lens, new_lens)):
        c, n = max(int(c), 0), max(int(n), 0)
        held, total = -(-c // page), -(-(c + n) // page)
        fits = total <= table.shape[1] and c + n < 2 ** 31
        need = total - held if fits else 0
        ok = fits and (need == 0 or at + need <= len(free_pages)) and row + n <= tokens
        if ok:
            table[i, held:total] = free_pages[at:at + need]
            for t in range(n):
                pg = table[i, (c + t) // page]
                if pg >= 0:
                    slots[row + t] = pg * page + (c + t) % page
                    positions[row + t] = c + t
            used += need
        else:
            refused += 1
        at += need
        row += n
        cu.append(min(row, tokens))
        kv.append(c + n if ok else c)
    return table, slots, positions, np.array(cu), np.array(kv, dtype=np.int64), np.array([used, refused])


def cover_code(amax) -> np.ndarray:
    """Least E8M0 code c >= 0 with amax <= 448 * 2^(c-127); 0 for amax 0 (fp64, exact)."""
    a = np.asarray(amax, dtype=np.float64)
    fr, ex = np.frexp(np.where(a > 0, a, 1.0))               # a = fr 2^ex, 448 = 7/8 2^9
    c = ex.astype(np.int64) - 9 + 127 + (fr > 0.875)
    return np.where(a > 0, np.maximum(c, 0), 0)


def _codes(x64, c):
    """E4M3 codes of x * 2^(127-c).  The product is rounded to fp32 once, which
    cannot change a code: fp32 holds it unless it is far below 2^-10."""
    with np.errstate(over="ignore", under="ignore", invalid="ignore"):
        return e4m3_from_f32(np.ldexp(x64, 127 - np.asarray(c)).astype(np.float32))


def append(x, slots, codes, scales, values: bool):
    """x [T, H, D] (fp32, or bf16 widened) into copies of codes and scales;
    `values` selects the transposed layout.  Returns (codes, scales)."""
    codes, scales = codes.copy(), scales.copy()
    P = codes.shape[3] if values else codes.shape[2]
    N = codes.shape[0]
    T = len(slots)
    t = 0
    while t < T:
        if not 0 <= slots[t] < N * P:
            t += 1
            continue
        z = t + 1
        while z < T and slots[z] == slots[z - 1] + 1 and slots[z] % P:
            z += 1
        pg, off = int(slots[t] // P), int(slots[t] % P)
        run = np.asarray(x[t:z], dtype=np.float64)           # [n, H, D]
        a = np.abs(run)
        c = cover_code(np.where(np.isfinite(a), a, 0).max(axis=(0, 2)))
        view = codes[pg].transpose(0, 2, 1) if values else codes[pg]     # [H, P, D]
        if off:
            old = scales[pg].astype(np.int64)
            c = np.maximum(c, old)
            moved = _codes(e4m3_decode(view[:, :off]), (127 + c - old)[:, None, None])
            view[:, :off] = np.where((c > old)[:, None, None], moved, view[:, :off])
        view[:, off:off + z - t] = _codes(run, c[None, :, None]).transpose(1, 0, 2)
        scales[pg] = c
        t = z
    return codes, scales


def attention(q, cu_q, kv_lens, k_codes, k_scales, v_codes, v_scales, table, sm_scale, softcap=0.0, window=0):
    """fp64 causal attention.  q [T, Hq, D] float64.  Returns (out, lse, weight,
    spread): weight[t, h] = sum_j w_j |v_j|, the scale of what rounding the
    probabilities may change, and spread[t, h] = max_j sum_d |q_d k_jd| *
    sm_scale, the scale of what rounding inside the scores may change.  Rows
    without a request are NaN."""
    N, H, P, D = k_codes.shape
    T, Hq, _ = q.shape
    G = Hq // H
    out = np.full((T, Hq, D), np.nan)
    lse = np.full((T, Hq), np.nan)
    weight = np.full((T, Hq, D), np.nan)
    spread = np.zeros((T, Hq))
    for i in range(len(kv_lens)):
        r0, r1 = int(cu_q[i]), int(cu_q[i + 1])
        m = min(int(kv_lens[i]), table.shape[1] * P)
        pages = np.asarray(table[i, :-(-m // P)], dtype=np.int64) if m > 0 else np.zeros(0, np.int64)
        good = (pages >= 0) & (pages < N)
        safe = np.where(good, pages, 0)
        there = np.repeat(good, P)[:max(m, 0)]
        for h in range(H):
            if m > 0:
                k = e4m3_decode(k_codes[safe, h]) * e8m0_decode(k_scales[safe, h])[:, None, None]
                v = e4m3_decode(v_codes[safe, h]).transpose(0, 2, 1) * e8m0_decode(v_scales[safe, h])[:, None, None]
                k, v = k.reshape(-1, D)[:m], v.reshape(-1, D)[:m]
            for t in range(r0, r1):
                pos = m - (r1 - r0) + (t - r0)
                lo = max(0, pos - window + 1) if window else 0
                seen = np.nonzero(there[lo:pos + 1])[0] + lo if pos >= 0 and m > 0 else np.zeros(0, np.int64)
                for g in range(h * G, h * G + G):
                    if len(seen) == 0:
                        out[t, g], lse[t, g], weight[t, g] = 0.0, -np.inf, 0.0
                        continue
                    s = (k[seen] @ q[t, g]) * sm_scale
                    spread[t, g] = (np.abs(k[seen]) @ np.abs(q[t, g])).max() * sm_scale
                    if softcap:
                        s = softcap * np.tanh(s / softcap)
                    top = s.max()
                    w = np.exp(s - top)
                    lse[t, g] = top + np.log(w.sum())
                    w /= w.sum()
                    out[t, g] = w @ v[seen]
                    weight[t, g] = w @ np.abs(v[seen])
    return out, lse, weight, spread
