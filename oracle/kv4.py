"""The 4-bit key/value cache (E2M1 elements, one E8M0 scale per 32 channels of
a token and head), the rotation by position that the append applies, and
causal attention over the pages.

Layouts: k_codes [N, H, P, D/2], v_codes [N, H, D/2, P] (uint8, channel 2j in the
low nibble of byte j), scales [N, H, D/32, P] (uint8 E8M0).  Codes and scales
of a token are those of `quantize_mxfp4` with block 32; what that leaves out is
settled here: scales are at most 252 (every value is finite), infinities
become 6 and NaN 0.  Derived from the formats alone: parity unpinned.
"""
from __future__ import annotations

import numpy as np

from .formats import E2M1_GRID, e8m0_decode
from .mxfp4 import e2m1_from_f64, pack_nibbles, quantize_mxfp4, unpack_nibbles

TOP = 252


def quantize(x):
    """x [..., D] fp32 -> (packed codes [..., D/2], scales [..., D/32])."""
    x = np.asarray(x, dtype=np.float32)
    b = x.reshape(-1, 32).astype(np.float64)
    fin = np.where(np.isfinite(b), b, 0.0)
    _, c = quantize_mxfp4(fin.astype(np.float32), 32)
    c = np.minimum(c, TOP)
    v = np.where(np.isnan(b), 0.0, np.clip(b, -4e38, 4e38)) * np.exp2(127.0 - c.astype(np.float64))
    codes = e2m1_from_f64(v, (np.signbit(b) & ~np.isnan(b)).astype(np.uint8))
    return pack_nibbles(codes.reshape(x.shape)), c.reshape(*x.shape[:-1], -1)


def append(x, slots, codes, scales, values: bool):
    """x [T, H, D] fp32 into copies of codes and scales; `values`: the transposed layout."""
    codes, scales = codes.copy(), scales.copy()
    P, N = scales.shape[3], scales.shape[0]
    new, c = quantize(x)
    for t, s in enumerate(slots):
        if 0 <= s < N * P:
            pg, off = int(s // P), int(s % P)
            if values:
                codes[pg, :, :, off] = new[t]
            else:
                codes[pg, :, off] = new[t]
            scales[pg, :, :, off] = c[t]
    return codes, scales


def rotate(x, positions, cos_sin, interleaved: bool):
    """x [T, H, D] turned by the angles of its positions, in fp64 (pair by pair)."""
    out = np.array(x, dtype=np.float64)
    half = cos_sin.shape[1] // 2
    for t, p in enumerate(positions):
        if not 0 <= p < len(cos_sin):
            continue
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            c, s = float(cos_sin[p, i]), float(cos_sin[p, half + i])
            u, v = out[t, :, a].copy(), out[t, :, b].copy()
            out[t, :, a] = u * c - v * s
            out[t, :, b] = v * c + u * s
    return out


def dequant(codes, scales, values: bool):
    """The cache as values [N, H, P, D] (fp64)."""
    if values:
        codes = codes.transpose(0, 1, 3, 2)
    n = unpack_nibbles(codes)
    v = E2M1_GRID[n & 7] * np.where(n & 8, -1.0, 1.0)
    return v * np.repeat(e8m0_decode(np.minimum(scales, TOP)).transpose(0, 1, 3, 2), 32, axis=3)


def attention(q, cu_q, kv_lens, k_codes, k_scales, v_codes, v_scales, table, sm_scale, softcap=0.0, window=0):
    """As `oracle.kv.attention` (same results: out, lse, weight, spread), on this cache."""
    N, H, P, _ = k_codes.shape
    T, Hq, D = q.shape
    G = Hq // H
    out, weight = np.full((T, Hq, D), np.nan), np.full((T, Hq, D), np.nan)
    lse, spread = np.full((T, Hq), np.nan), np.zeros((T, Hq))
    kv, vv = dequant(k_codes, k_scales, False), dequant(v_codes, v_scales, True)
    for i in range(len(kv_lens)):
        r0, r1 = int(cu_q[i]), int(cu_q[i + 1])
        m = max(0, min(int(kv_lens[i]), table.shape[1] * P))
        pages = np.asarray(table[i, :-(-m // P)], dtype=np.int64)
        good = (pages >= 0) & (pages < N)
        there = np.repeat(good, P)[:m]
        safe = np.where(good, pages, 0)
        for h in range(H):
            k, v = kv[safe, h].reshape(-1, D)[:m], vv[safe, h].reshape(-1, D)[:m]
            for t in range(r0, r1):
                pos = m - (r1 - r0) + (t - r0)
                lo = max(0, pos - window + 1) if window else 0
                seen = np.nonzero(there[lo:pos + 1])[0] + lo if pos >= 0 else np.zeros(0, np.int64)
                rows = slice(h * G, h * G + G)
                if len(seen) == 0:
                    out[t, rows], lse[t, rows], weight[t, rows] = 0.0, -np.inf, 0.0
                    continue
                s = (q[t, rows] @ k[seen].T) * sm_scale
                spread[t, rows] = (np.abs(q[t, rows]) @ np.abs(k[seen]).T).max(1) * sm_scale
                if softcap:
                    s = softcap * np.tanh(s / softcap)
                top = s.max(1, keepdims=True)
                w = np.exp(s - top)
                total = w.sum(1, keepdims=True)
                lse[t, rows] = (top + np.log(total))[:, 0]
                out[t, rows] = (w / total) @ v[seen]
                weight[t, rows] = (w / total) @ np.abs(v[seen])
    return out, lse, weight, spread
