"""GPU parity of the 4-bit key/value cache (append, attention) and of the append
that rotates by position, with the oracle: codes and scales bit for bit,
attention within the bound on its roundings of the 8-bit cache (`_bounds`)."""
import numpy as np
import pytest
import torch

from oracle import kv as OK
from oracle import kv4 as O4
from oracle.formats import bf16_decode, bf16_round
from tests.gpu_helpers import banner, dev_bf16, dev_f32, dev_u8, host_bits16, host_f32, host_u8
from tests.test_gpu_kv import SHAPES, W, _bounds, _cache, _i32, _i64, _np, _slots  # noqa: F401 (W is a fixture)

pytestmark = pytest.mark.gpu


def _cache4(g, N, H, P, D, lo=118, hi=131):
    """Random codes, scales around 1."""
    return [g.integers(0, 256, (N, H, P, D // 2)).astype(np.uint8), g.integers(lo, hi, (N, H, D // 32, P)).astype(np.uint8),
            g.integers(0, 256, (N, H, D // 2, P)).astype(np.uint8), g.integers(lo, hi, (N, H, D // 32, P)).astype(np.uint8)]


def _dev(x, bf16):
    """(device tensor, the fp32 values it holds)."""
    if bf16:
        b = bf16_round(x)
        return dev_bf16(b), bf16_decode(b).astype(np.float32)
    return dev_f32(x), np.asarray(x, np.float32)


def _same(dev, want):
    for name, d, w in zip(("keys", "key scales", "values", "value scales"), dev, want):
        assert np.array_equal(host_u8(d), w), name


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
def _check_append(W, k, v, slots, cache, bf16):
    dev = [dev_u8(c) for c in cache]
    (kd, k), (vd, v) = _dev(k, bf16), _dev(v, bf16)
    W.wq_kv4_append(kd, vd, _i64(slots), *dev)
    _same(dev, (*O4.append(k, slots, *cache[:2], False), *O4.append(v, slots, *cache[2:], True)))


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("H,D,page,ctx,new", [
    (1, 64, 16, [0], [1]),
    (8, 128, 64, list(range(0, 640, 10)), [1] * 64),       # a decode step
    (2, 128, 16, [3, 0, 16, 31], [40, 16, 1, 2]),
    (3, 64, 32, [5, 0, 0], [100, 0, 333]),
    (1, 128, 128, [100, 1], [300, 126]),
    (5, 128, 64, [63, 1], [700, 62]),
    (16, 64, 128, [7], [3500]),                            # chunks of 64 tokens
])
def test_append(W, bf16, H, D, page, ctx, new):
    banner("kv4 append", bf16, H, D, page, ctx[:4], new[:4])
    g = np.random.default_rng(H * D + page + len(ctx))
    slots, N = _slots(g, ctx, new, page, spare=2)
    T = len(slots)
    amp = np.exp2(g.integers(-12, 12, (T, H, 1)))
    k, v = ((g.standard_normal((T, H, D)) * amp).astype(np.float32) for _ in range(2))
    _check_append(W, k, v, slots, _cache4(g, N, H, page, D), bf16)


@pytest.mark.parametrize("T,H", [(50, 2), (900, 8)])
def test_append_slots_in_any_order(W, T, H):
    """Neighbouring tokens anywhere, also backwards and with gaps inside a page, and slots outside the cache."""
    banner("kv4 append: slots in any order", T, H)
    g = np.random.default_rng(T)
    P, D, N = 16, 64, 80
    slots = g.permutation(1200)[:T]                        # pages 75 to 79 are for the ones by hand
    slots[:8] = np.arange(1200, 1208)[::-1]
    slots[8:20] = [-1, N * P, 1 << 40, -(1 << 62), 1240, 1241, 1242, 1243, 1244, 1246, 1247, 1248]
    k, v = (g.standard_normal((T, H, D)).astype(np.float32) for _ in range(2))
    _check_append(W, k, v, slots, _cache4(g, N, H, P, D), True)


def _special(g, T, H, D):
    x = g.standard_normal((T, H, D)).astype(np.float32)
    x[0] = 0.0
    x[1] = -0.0
    x[2, 0, :4] = [np.nan, -np.nan, np.inf, -np.inf]
    x[3] = np.nan
    x[4] = np.inf
    x[5] = np.clip(x[5], -1, 1) * 3e38
    x[6] *= 1e-38
    x[7] *= 2.0 ** -140                                    # fp32 subnormals
    # midpoints of the grid at a scale of 1 (the block's 6 sets it)
    x[8, 0, :32] = np.concatenate([[6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], -np.linspace(0, 6, 24)])
    return np.clip(x, -3.38e38, 3.38e38, where=np.isfinite(x), out=x)


@pytest.mark.parametrize("bf16", [True, False])
def test_append_special_values(W, bf16):
    banner("kv4 append: zeros, NaN, infinities, extremes, ties", bf16)
    g = np.random.default_rng(3)
    H, D, P = 1, 64, 16
    k, v = _special(g, 12, H, D), _special(g, 12, H, D)[::-1].copy()
    slots = np.array([0, 17, 2 * P + 15, 3 * P, 4 * P, 5 * P, 6 * P, 7 * P + 3, 8 * P, 9 * P, 10 * P, 11 * P + 15])
    _check_append(W, k, v, slots, _cache4(g, 12, H, P, D), bf16)


# ---------------------------------------------------------------------------
# rotation
# ---------------------------------------------------------------------------
def _angles(max_pos, rot):
    a = np.arange(max_pos, dtype=np.float64)[:, None] * 10000.0 ** -(np.arange(0, rot, 2) / rot)
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def _check_rotary(W, q, k, v, pos, cs, slots, cache, bf16, inter, in_place=False):
    """Keys and values bit for bit as the appends store the rotated keys, rounded once to fp32;
    queries within half a bf16 step and the two fp32 roundings of a a cos + b sin."""
    eight = cache[1].ndim == 2
    dev = [dev_u8(c) for c in cache]
    (kd, k), (vd, v) = _dev(k, bf16), _dev(v, bf16)
    live = (pos >= 0) & (pos < len(cs))
    qd = out = None
    if q is not None:
        qd, q = _dev(q, bf16)
        out = qd if in_place else torch.full(qd.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    got = W.wq_kv_append_rotary(qd, kd, vd, _i32(pos), dev_f32(cs), _i64(slots), *dev, interleaved=inter, q_out=out)
    kr = O4.rotate(k, pos, cs, inter).astype(np.float32)
    sl = np.where(live, slots, -1)
    ap = OK.append if eight else O4.append
    _same(dev, (*ap(kr, sl, *cache[:2], False), *ap(v, sl, *cache[2:], True)))
    if q is None:
        assert got is None
        return
    assert got is out
    y, want = bf16_decode(host_bits16(got)), O4.rotate(q, pos, cs, inter)
    size = O4.rotate(np.abs(q).astype(np.float64), pos, np.abs(cs), inter)  # |a||cos| - |b||sin|: not the bound, so
    size = np.abs(size) + 2 * np.abs(q).max(-1, keepdims=True)              # with room: every term is below the row's largest
    assert (np.abs(y - want)[live] <= (2.0 ** -8 * np.abs(want) + 2.0 ** -22 * size)[live]).all()
    before = q if in_place else np.full_like(q, 7.0)
    assert np.array_equal(y[~live], before[~live]), "rows without a position changed"


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("Hq,H,D,page,rot,inter,ctx,new", [
    (1, 1, 64, 16, 64, False, [0], [1]),
    (32, 8, 128, 64, 128, False, list(range(0, 640, 10)), [1] * 64),   # a decode step
    (8, 2, 128, 16, 128, True, [3, 0, 16, 31], [40, 16, 1, 2]),
    (3, 3, 64, 32, 16, False, [5, 0, 0], [100, 0, 333]),               # a part of the channels
    (4, 1, 128, 128, 48, True, [100, 1], [300, 126]),
    (5, 5, 128, 64, 96, False, [63, 1], [700, 62]),
])
def test_append_rotary(W, bits, bf16, Hq, H, D, page, rot, inter, ctx, new):
    banner("kv append rotary", bits, bf16, Hq, H, D, page, rot, inter, ctx[:4], new[:4])
    g = np.random.default_rng(Hq * D + page + rot)
    slots, N = _slots(g, ctx, new, page, spare=2)
    T = len(slots)
    cs = _angles(900, rot)
    pos = np.concatenate([c + np.arange(n) for c, n in zip(ctx, new)] + [[-1, -1]])
    amp = np.exp2(g.integers(-3, 4, (T, H, 1)))
    k, v = ((g.standard_normal((T, H, D)) * amp).astype(np.float32) for _ in range(2))
    q = g.standard_normal((T, Hq, D)).astype(np.float32)
    cache = _cache4(g, N, H, page, D) if bits == 4 else _cache(g, N, H, page, D)
    _check_rotary(W, q, k, v, pos, cs, slots, cache, bf16, inter)
    if bf16:
        _check_rotary(W, q, k, v, pos, cs, slots, cache, bf16, inter, in_place=True)
    else:
        _check_rotary(W, None, k, v, pos, cs, slots, cache, bf16, inter)


@pytest.mark.parametrize("bits", [8, 4])
def test_append_rotary_positions_outside_the_table(W, bits):
    """Tokens in the middle of a run whose position has no angles are left out of the cache and of q_out."""
    banner("kv append rotary: positions without angles", bits)
    g = np.random.default_rng(5)
    H, D, P, T = 2, 64, 16, 40
    pos = np.arange(T)
    pos[[3, 16, 17, 30]] = [-1, 64, 1 << 30, -(1 << 31)]
    slots, N = _slots(g, [0], [T], P)
    slots[30:] = -1                                        # two runs on a page are outside the 8-bit contract
    slots[0:4], slots[16:18] = -1, slots[16:18]
    k, v = (g.standard_normal((T, H, D)).astype(np.float32) for _ in range(2))
    q = g.standard_normal((T, 4, D)).astype(np.float32)
    cache = _cache4(g, N, H, P, D) if bits == 4 else _cache(g, N, H, P, D)
    _check_rotary(W, q, k, v, pos, _angles(64, 64), slots, cache, True, False)


@pytest.mark.parametrize("bits", [8, 4])
def test_append_rotary_special_values(W, bits):
    """NaN and infinite keys, and angles of zero, whose rotation is the identity."""
    banner("kv append rotary: NaN, infinities, extremes at angle 0", bits)
    g = np.random.default_rng(6)
    H, D, P, T = 1, 64, 16, 12
    k, v = _special(g, T, H, D), _special(g, T, H, D)[::-1].copy()
    k[2, 0, 4:8] = 0.0
    slots = np.arange(T) * P
    cs = np.zeros((T, D), np.float32)
    cs[:, :D // 2] = 1.0
    # NaN and infinity times the sine of zero are NaN: the partner is NaN too, and so is the pair
    cache = _cache4(g, T, H, P, D) if bits == 4 else _cache(g, T, H, P, D)
    with np.errstate(invalid="ignore"):
        kr = O4.rotate(k, np.arange(T), cs, False).astype(np.float32)
    dev = [dev_u8(c) for c in cache]
    W.wq_kv_append_rotary(None, dev_f32(k), dev_f32(v), _i32(np.arange(T)), dev_f32(cs), _i64(slots), *dev)
    ap = OK.append if bits == 8 else O4.append
    want = [*ap(kr, slots, *cache[:2], False), *ap(v, slots, *cache[2:], True)]
    got = [host_u8(d) for d in dev]
    if bits == 8:                                          # the sign of a NaN that arithmetic makes is open
        for x in (got, want):
            x[0] = np.where((x[0] & 0x7F) == 0x7F, 0x7F, x[0])
    for name, d, w in zip(("keys", "key scales", "values", "value scales"), got, want):
        assert np.array_equal(d, w), name


def test_append_rotary_is_the_append_of_rotated_keys(W):
    """The 8-bit cache after the rotating append, and after the plain append of keys rotated beforehand."""
    banner("kv append rotary: against the plain append")
    g = np.random.default_rng(7)
    H, D, P = 4, 128, 64
    slots, N = _slots(g, [5, 64], [130, 40], P)
    T = len(slots)
    pos = np.concatenate([5 + np.arange(130), 64 + np.arange(40)])
    k, v = (g.standard_normal((T, H, D)).astype(np.float32) for _ in range(2))
    cs = _angles(300, D)
    for bits in (8, 4):
        cache = _cache4(g, N, H, P, D) if bits == 4 else _cache(g, N, H, P, D)
        a, b = ([dev_u8(c) for c in cache] for _ in range(2))
        W.wq_kv_append_rotary(None, dev_f32(k), dev_f32(v), _i32(pos), dev_f32(cs), _i64(slots), *a)
        kr = O4.rotate(k, pos, cs, False).astype(np.float32)
        (W.wq_kv4_append if bits == 4 else W.wq_kv_append)(dev_f32(kr), dev_f32(v), _i64(slots), *b)
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("bits", [8, 4])
def test_append_rotary_strided_in_place(W, bits):
    """Queries, keys and values as slices of one projection's rows, the queries turned where they lie."""
    banner("kv append rotary: slices of one projection, in place", bits)
    g = np.random.default_rng(8)
    Hq, H, D, P, T = 6, 2, 64, 16, 70
    slots, N = _slots(g, [5], [T], P)
    width = (Hq + 2 * H) * D
    b = bf16_round(g.standard_normal((T, width)))
    x = bf16_decode(b).astype(np.float32)
    fused = dev_bf16(b)
    q, k, v = (fused[:, a * D:z * D].view(T, -1, D) for a, z in ((0, Hq), (Hq, Hq + H), (Hq + H, Hq + 2 * H)))
    cache = _cache4(g, N, H, P, D) if bits == 4 else _cache(g, N, H, P, D)
    dev = [dev_u8(c) for c in cache]
    cs, pos = _angles(100, 32), 5 + np.arange(T)
    W.wq_kv_append_rotary(q, k, v, _i32(pos), dev_f32(cs), _i64(slots), *dev, q_out=q)
    xk = x[:, Hq * D:(Hq + H) * D].reshape(T, H, D)
    ap = OK.append if bits == 8 else O4.append
    _same(dev, (*ap(O4.rotate(xk, pos, cs, False).astype(np.float32), slots, *cache[:2], False),
                *ap(x[:, (Hq + H) * D:].reshape(T, H, D), slots, *cache[2:], True)))
    y = bf16_decode(host_bits16(fused))
    assert np.array_equal(y[:, Hq * D:], x[:, Hq * D:]), "keys and values stay as they were"
    want = O4.rotate(x[:, :Hq * D].reshape(T, Hq, D), pos, cs, False).reshape(T, -1)
    assert (np.abs(y[:, :Hq * D] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -21 * np.abs(x).max()).all()


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def _problem(seed, Hq, H, D, P, q_lens, kv_lens, spare_rows=0, spare_cols=1):
    g = np.random.default_rng(seed)
    held = [-(-m // P) for m in kv_lens]
    N = sum(held) + 2
    ids = g.permutation(N)
    table = np.full((len(kv_lens), max(held, default=0) + spare_cols), -1)
    at = 0
    for i, n in enumerate(held):
        table[i, :n] = ids[at:at + n]
        at += n
    q = g.standard_normal((int(sum(q_lens)) + spare_rows, Hq, D)) * 0.5
    return q, np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int64), list(kv_lens), _cache4(g, N, H, P, D), table


def _poison(cache, table, kv):
    """Copies in which what the call must not use has the largest codes and the NaN scale."""
    cache = [c.copy() for c in cache]
    N, P = cache[1].shape[0], cache[1].shape[3]
    used = np.zeros((N, P), bool)
    for i, m in enumerate(kv):
        for j in range(0, min(int(m), table.shape[1] * P)):
            pg = table[i][j // P]
            if 0 <= pg < N:
                used[pg, j % P] = True
    free = ~used
    cache[0].transpose(0, 2, 1, 3)[free] = 0x7F
    for c in (1, 3):
        cache[c].transpose(0, 3, 1, 2)[free] = 255
    cache[2].transpose(0, 3, 1, 2)[free] = 0xF7
    return cache


def _check_attention(W, q, cu, kv, cache, table, poison=True, **kw):
    T, Hq, D = q.shape
    P = cache[1].shape[3]
    bits = bf16_round(q)
    opts = {"sm_scale": D ** -0.5, "softcap": 0.0, "window": 0}
    opts.update({k: kw[k] for k in opts if k in kw})
    ref, lse, weight, spread = O4.attention(bf16_decode(bits), cu, kv, *cache, table, **opts)
    if poison:
        cache = _poison(cache, table, kv)
    out = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    got, glse = W.wq_kv4_attention(dev_bf16(bits), *[dev_u8(c) for c in cache], _i32(table), _i32(cu), _i32(kv),
                                   out=out, return_lse=True, **kw)
    torch.cuda.synchronize()
    y, l = bf16_decode(host_bits16(got)), host_f32(glse).astype(np.float64)
    real = ~np.isnan(ref[:, 0, 0])
    assert (y[~real] == 7.0).all(), "rows behind the last request changed"
    seen = max(1, min(int(max(kv, default=1)), table.shape[1] * P))
    # a capped score is off by at most softcap * 2^-22 more
    tol, tol_lse = _bounds(ref[real], weight[real], spread[real] + opts["softcap"] * 2.0 ** -22 / ((D + 16) * 2.0 ** -24),
                           seen, D)
    assert np.isfinite(y[real]).all()
    worst = (np.abs(y[real] - ref[real]) / tol).max(initial=0.0)
    assert worst <= 1.0, f"output: error / bound = {worst:.3f}"
    none = np.isneginf(lse[real])
    assert np.array_equal(none, np.isneginf(l[real]))
    with np.errstate(invalid="ignore"):
        d = np.where(none, 0.0, np.abs(l[real] - lse[real]) / (tol_lse + 2.0 ** -22 * np.abs(lse[real])))
    assert d.max(initial=0.0) <= 1.0, f"lse: error / bound = {d.max():.3f}"
    return got


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}x{s[1]}x{s[2]}p{s[3]}")
@pytest.mark.parametrize("hint", [0, 1, "max"])
def test_attention(W, shape, hint):
    Hq, H, D, P, ql, kl = shape
    banner("kv4 attention", shape, hint)
    q, cu, kv, cache, table = _problem(1, Hq, H, D, P, ql, kl, spare_rows=3)
    _check_attention(W, q, cu, kv, cache, table, max_q=max(ql) if hint == "max" else hint)


@pytest.mark.parametrize("shape", SHAPES[1:], ids=lambda s: f"{s[0]}x{s[1]}x{s[2]}p{s[3]}")
@pytest.mark.parametrize("softcap,window", [(0.0, 1), (0.0, 50), (5.0, 0), (20.0, 64), (0.0, 100000)])
def test_attention_window_and_cap(W, shape, softcap, window):
    Hq, H, D, P, ql, kl = shape
    banner("kv4 attention window / cap", shape, softcap, window)
    q, cu, kv, cache, table = _problem(2, Hq, H, D, P, ql, kl)
    _check_attention(W, q, cu, kv, cache, table, softcap=softcap, window=window, sm_scale=0.02)


@pytest.mark.parametrize("ql", [[1, 1, 1, 1], [40, 3, 150, 1]])
def test_attention_rows_that_see_nothing(W, ql):
    """No cache at all, fewer tokens than queries, a window on pages that are not there."""
    banner("kv4 attention: rows without a token", ql)
    kl = [0, 2, 20, 33]
    q, cu, kv, cache, table = _problem(3, 8, 2, 64, 16, ql, kl)
    _check_attention(W, q, cu, kv, cache, table)
    table[3, 2] = -1
    table[2, 0] = len(cache[1])
    _check_attention(W, q, cu, kv, cache, table)
    _check_attention(W, q, cu, kv, cache, table, window=1)


@pytest.mark.parametrize("D,P", [(128, 16), (64, 32), (128, 64)])
@pytest.mark.parametrize("ql", [[1, 1], [90, 2]])
def test_attention_pages_that_are_not_there(W, ql, D, P):
    banner("kv4 attention: page ids outside the cache", ql, D, P)
    q, cu, kv, cache, table = _problem(4, 4, 2, D, P, ql, [18 * P + 12, 10 * P + 10])
    table[0, [0, 3, 4, 9]] = [-1, 1 << 30, -(1 << 31), len(cache[1])]
    table[1, 10] = -5
    _check_attention(W, q, cu, kv, cache, table)


def test_attention_lengths_outside_the_contract(W):
    """Lengths past the table, negative ones and row ranges past the arrays are clamped."""
    banner("kv4 attention: lengths and ranges that do not fit")
    q, cu, kv, cache, table = _problem(5, 4, 2, 64, 16, [2, 3, 1, 2], [40, 20, 9, 30], spare_cols=0)
    got = _check_attention(W, q, cu, [1000, -7, 9, 30], cache, table, poison=False)
    assert got.shape[0] == 8
    for bad in ([0, 2, 5, 4, 100], [-3, 2, 5, 6, 8], [0, 2 ** 31 - 1, 5, 6, 8], [5, 4, 3, 2, 1]):
        for hint in (0, 1):
            out = W.wq_kv4_attention(dev_bf16(bf16_round(q)), *[dev_u8(c) for c in cache], _i32(table), _i32(bad),
                                     _i32(kv), max_q=hint)
            torch.cuda.synchronize()
            assert out.shape == q.shape


@pytest.mark.parametrize("ql", [[1, 3, 1], [70, 3, 130]])
def test_attention_shared_pages_and_far_scales(W, ql):
    """Two requests on the same first pages; scales of neighbouring tokens and blocks apart by 2^40."""
    banner("kv4 attention: shared prefix, far scales", ql)
    q, cu, kv, cache, table = _problem(6, 8, 2, 128, 32, ql, [100, 130, 200])
    table[1, :3] = table[0, :3]
    table[2, :2] = table[0, :2]
    g = np.random.default_rng(6)
    cache[3][:] = g.integers(100, 141, cache[3].shape)
    cache[1][:] = g.integers(90, 121, cache[1].shape)
    _check_attention(W, q, cu, kv, cache, table, poison=False)


@pytest.mark.parametrize("ql", [[1, 1], [70, 3]])
def test_attention_extreme_scales(W, ql):
    """Value scales of 2^-127 beside 1; values up to 6 * 2^100 (the tokens that see no such one stay exact)."""
    banner("kv4 attention: scales at the ends of their range", ql)
    q, cu, kv, cache, table = _problem(16, 4, 2, 64, 16, ql, [90, 40])
    g = np.random.default_rng(16)
    cache[3][:] = g.choice([0, 1, 60, 127], cache[3].shape)
    _check_attention(W, q, cu, kv, cache, table)
    cache[3][:] = 0
    cache[3][:, :, 0] = g.choice([0, 227], cache[3][:, :, 0].shape)
    _check_attention(W, q, cu, kv, cache, table)


def test_attention_extreme_scores(W):
    """Scores of some thousands: one token takes everything, in the first or the last tile."""
    banner("kv4 attention: peaked scores")
    for seed in range(2):
        q, cu, kv, cache, table = _problem(7 + seed, 4, 1, 64, 16, [1, 20], [333, 500])
        q *= 4000
        if seed:
            cache[1][:] = 127
        _check_attention(W, q, cu, kv, cache, table, sm_scale=1e-1)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ql", [[1, 3, 1], [40, 1, 90]])
@pytest.mark.parametrize("softcap,sm_scale", [(2.0, 1.0), (30.0, 0.5), (1000.0, 0.05), (0.002, 0.01), (50.0, 1e-4)])
def test_attention_caps(W, D, ql, softcap, sm_scale):
    """Scores far above their cap and far below it, in one tile and apart."""
    banner("kv4 attention: caps", D, ql, softcap, sm_scale)
    q, cu, kv, cache, table = _problem(17, 8, 2, D, 16, ql, [300, 70, 500])
    _check_attention(W, q, cu, kv, cache, table, softcap=softcap, sm_scale=sm_scale)


def test_attention_strided_queries(W):
    banner("kv4 attention: queries as slices of wider rows")
    q, cu, kv, cache, table = _problem(9, 8, 2, 64, 16, [1, 40, 3], [50, 40, 9])
    bits = bf16_round(q)
    wide = torch.zeros((q.shape[0], 3 * 8 * 64), dtype=torch.bfloat16, device="cuda")
    mid = wide[:, 512:1024].view(-1, 8, 64)
    mid.copy_(dev_bf16(bits))
    dev = [dev_u8(c) for c in cache]
    args = (*dev, _i32(table), _i32(cu), _i32(kv))
    a, b = W.wq_kv4_attention(mid, *args), W.wq_kv4_attention(dev_bf16(bits), *args)
    assert torch.equal(a, b)


def test_attention_one_long_context_beside_short_ones(W):
    banner("kv4 attention: 20000 tokens beside short contexts")
    q, cu, kv, cache, table = _problem(10, 4, 2, 64, 64, [1, 1, 1, 2], [20000, 3, 900, 5000])
    _check_attention(W, q, cu, kv, cache, table, poison=False)


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("H,group,most_q,D", [(8, 2, 1, 64), (8, 4, 6, 64), (5, 3, 1, 128), (16, 2, 10, 128), (3, 16, 4, 64)])
def test_attention_shares_over_requests(W, page, H, group, most_q, D):
    """Ragged batches whose tiles are cut into shares that begin and end anywhere: several requests to
    a wave, several waves to a request, requests without rows or without a cache between them."""
    banner("kv4 attention: shares over requests", page, H, group, most_q, D)
    g = np.random.default_rng(H + page)
    kl = np.exp(g.uniform(0, np.log(3000), 40)).astype(int)
    ql = g.integers(1, most_q + 1, 40)
    kl[[3, 17]], ql[[5, 6, 30]], kl[[9, 22]] = 0, 0, [2999, 2048]
    q, cu, kv, cache, table = _problem(14, H * group, H, D, page, ql, kl, spare_rows=2)
    for kw in ({}, {"window": 700}):
        _check_attention(W, q, cu, kv, cache, table, max_q=most_q, **kw)


@pytest.mark.parametrize("hint", [0, 1])
def test_attention_many_short_requests(W, hint):
    banner("kv4 attention: 900 requests of a few tokens, 16 key heads", hint)
    g = np.random.default_rng(15)
    kl, ql = g.integers(0, 130, 900), g.integers(0, 3, 900)
    q, cu, kv, cache, table = _problem(15, 16, 16, 64, 16, ql, kl)
    _check_attention(W, q, cu, kv, cache, table, max_q=2 if hint else 0)


@pytest.mark.parametrize("page", [32, 64])
def test_attention_chunk_of_a_long_prompt(W, page):
    """Few rows and many tokens: prompt tiles are split over the cache, beside short requests."""
    banner("kv4 attention: chunks of 40 and 90 rows on 3000 tokens", page)
    q, cu, kv, cache, table = _problem(18, 8, 2, 128, page, [40, 1, 90, 5], [3000, 700, 2500, 64])
    for kw in ({}, {"softcap": 10.0}, {"window": 1500}):
        _check_attention(W, q, cu, kv, cache, table, **kw)


@pytest.mark.parametrize("Hq,H,D,P,ql", [(8, 2, 128, 64, [1, 1, 1]), (4, 4, 64, 16, [1, 3, 2]), (8, 2, 64, 128, [5, 1, 4]),
                                         (8, 2, 128, 64, [90, 1, 40]), (4, 2, 64, 32, [130, 3, 70])])
@pytest.mark.parametrize("softcap", [0.0, 8.0])
def test_attention_does_not_depend_on_bytes_no_row_sees(W, Hq, H, D, P, ql, softcap):
    """The same bits whatever stands behind the last token, before the window and in pages of others."""
    banner("kv4 attention: unseen bytes", Hq, H, D, P, ql, softcap)
    q, cu, kv, cache, table = _problem(19, Hq, H, D, P, ql, [300, 131, 200])
    table[1, 1] = -1
    for window in (0, 60):
        got = []
        for c in (cache, _poison(cache, table, kv)):
            out, lse = W.wq_kv4_attention(dev_bf16(bf16_round(q)), *[dev_u8(x) for x in c], _i32(table), _i32(cu),
                                          _i32(kv), softcap=softcap, window=window, return_lse=True)
            got.append((out, lse))
        assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@pytest.mark.parametrize("ql", [[1, 7], [3, 90]])
def test_attention_rows_do_not_depend_on_tokens_behind_them(W, ql):
    """A token with the NaN scale, or with the largest values, changes nothing in the rows before it."""
    banner("kv4 attention: tokens that some rows of a tile do not see", ql)
    q, cu, kv, cache, table = _problem(20, 4, 2, 64, 16, ql, [50, 100])
    a = W.wq_kv4_attention(dev_bf16(bf16_round(q)), *[dev_u8(x) for x in cache], _i32(table), _i32(cu), _i32(kv))
    last = table[1, 99 // 16]
    for c in (255, 252):
        bad = [x.copy() for x in cache]
        bad[3][last, :, :, 99 % 16] = c
        bad[2][last, :, :, 99 % 16] = 0x7F
        if c == 255:
            bad[1][last, :, :, 99 % 16] = 255
        b = W.wq_kv4_attention(dev_bf16(bf16_round(q)), *[dev_u8(x) for x in bad], _i32(table), _i32(cu), _i32(kv))
        assert torch.equal(a[:-1], b[:-1])


def test_cache_past_32_bits(W):
    """Pages whose bytes lie beyond 2^32."""
    banner("kv4 attention and append: a cache of 4.6 GB codes each")
    N, H, P, D = 140000, 8, 64, 128
    kc = torch.empty((N, H, P, D // 2), dtype=torch.uint8, device="cuda")
    vc = torch.empty((N, H, D // 2, P), dtype=torch.uint8, device="cuda")
    ks, vs = (torch.empty((N, H, D // 32, P), dtype=torch.uint8, device="cuda") for _ in range(2))
    g = np.random.default_rng(11)
    pages = np.array([139999, 3, 131072, 80000])
    k, v = (bf16_round(g.standard_normal((200, H, D))) for _ in range(2))
    slots = np.concatenate([p * P + np.arange(P) for p in pages])[:200]
    cs, pos = _angles(200, D), np.arange(200)
    qb = bf16_round(g.standard_normal((200, 16, D)))
    qr = W.wq_kv_append_rotary(dev_bf16(qb), dev_bf16(k), dev_bf16(v), _i32(pos), dev_f32(cs), _i64(slots), kc, ks, vc, vs)
    small = [np.zeros((4, H, P, D // 2), np.uint8), np.zeros((4, H, D // 32, P), np.uint8),
             np.zeros((4, H, D // 2, P), np.uint8), np.zeros((4, H, D // 32, P), np.uint8)]
    at = np.concatenate([i * P + np.arange(P) for i in range(4)])[:200]
    kr = O4.rotate(bf16_decode(k).astype(np.float32), pos, cs, False).astype(np.float32)
    small[0], small[1] = O4.append(kr, at, small[0], small[1], False)
    small[2], small[3] = O4.append(bf16_decode(v).astype(np.float32), at, small[2], small[3], True)
    for q, cu in ((qr[197:], [0, 1, 3]), (qr, [0, 100, 200])):
        args = (_i32([[0, 1, 2, 3]] * 2), _i32(cu), _i32([150, 200]))
        a = W.wq_kv4_attention(q, *[dev_u8(c) for c in small], *args)
        b = W.wq_kv4_attention(q, kc, ks, vc, vs, _i32([pages] * 2), *args[1:])
        assert torch.equal(a, b)
    assert np.array_equal(host_u8(kc[_i64(pages[:3])]), small[0][:3])
    assert np.array_equal(host_u8(vc[_i64(pages[:3])]), small[2][:3])


# ---------------------------------------------------------------------------
# refusals, graphs, streams
# ---------------------------------------------------------------------------
def test_refusals_of_the_binding(W):
    banner("kv4: shapes and types the binding refuses")
    q, cu, kv, cache, table = _problem(12, 4, 2, 64, 16, [2], [20])
    x, c = dev_bf16(bf16_round(q)), [dev_u8(a) for a in cache]
    t, u, n = _i32(table), _i32(cu), _i32(kv)
    ok = lambda q=x, c=c, t=t, u=u, n=n, **kw: W.wq_kv4_attention(q, *c, t, u, n, **kw)
    ok()
    eight = [dev_u8(a) for a in _cache(np.random.default_rng(0), 4, 2, 16, 64)]
    for bad in (dict(q=x.float()), dict(q=x[:, :3].contiguous()), dict(q=x.transpose(0, 1)), dict(t=t.long()),
                dict(t=t[0]), dict(u=u[:1]), dict(n=n.repeat(2)), dict(n=n.cpu()), dict(c=c[:3] + [c[1].int()]),
                dict(c=[c[0], c[1], c[0], c[3]]), dict(c=eight), dict(softcap=-1.0), dict(window=-2), dict(sm_scale=0.0),
                dict(max_q=-1), dict(out=torch.empty_like(x)[:1]), dict(workspace=[0])):
        with pytest.raises(ValueError):
            ok(**bad)
    k = torch.zeros((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    s = _i64([0, 1])
    for bad in ((k[:, :1], k, s), (k, k.float(), s), (k.half(), k.half(), s), (k, k, s.int()), (k, k, s[:1])):
        with pytest.raises(ValueError):
            W.wq_kv4_append(*bad, *c)
    with pytest.raises(ValueError):
        W.wq_kv4_append(k, k, s, *eight)
    with pytest.raises(ValueError):
        W.wq_kv_append(k, k, s, *c)
    p, cs = _i32([0, 1]), torch.ones(4, 64, device="cuda")
    for cache in (c, eight):
        W.wq_kv_append_rotary(x, k, k, p, cs, s, *cache)
        for bad in (dict(q=x.float()), dict(q=x[:1]), dict(q=x[:, :, :32]), dict(pos=p.long()), dict(pos=p[:1]),
                    dict(cs=cs.double()), dict(cs=cs[0]), dict(cs=cs[:, :24].contiguous()), dict(cs=cs[:0]),
                    dict(cs=cs.cpu()), dict(s=s.int()), dict(out=x.float()), dict(out=x[:, :2]),
                    dict(q=None, out=x), dict(cs=torch.ones(4, 128, device="cuda"))):
            a = dict(q=x, pos=p, cs=cs, s=s, out=None)
            a.update(bad)
            with pytest.raises(ValueError):
                W.wq_kv_append_rotary(a["q"], k, k, a["pos"], a["cs"], a["s"], *cache, q_out=a["out"])


def _serve(W, steps, H, G, D, P, width, seed, rot, inter):
    """Prompts, then decode steps over a 4-bit cache: tables, rotating append, attention."""
    g = torch.Generator("cuda").manual_seed(seed)
    B = len(steps[0])
    N = B * width + 1
    kc = torch.full((N, H, P, D // 2), 0x77, dtype=torch.uint8, device="cuda")
    vc = torch.full((N, H, D // 2, P), 0x77, dtype=torch.uint8, device="cuda")
    ks, vs = (torch.full((N, H, D // 32, P), 255, dtype=torch.uint8, device="cuda") for _ in range(2))
    table = _i32(np.full((B, width), -1))
    free = torch.randperm(N, device="cuda", generator=g).int()
    ctx, cursor = _i32(np.zeros(B)), _i32([0])
    cs = dev_f32(_angles(width * P, rot))
    for new in steps:
        T = sum(new)
        slots, pos, cu, kv, state = W.wq_kv_blocks(ctx, _i32(new), free, table, P, T, cursor=cursor)
        qkv = torch.randn(T, (H * G + 2 * H) * D, device="cuda", generator=g).to(torch.bfloat16)
        q = qkv[:, :H * G * D].view(T, H * G, D)
        k = qkv[:, H * G * D:(H * G + H) * D].view(T, H, D)
        v = qkv[:, (H * G + H) * D:].view(T, H, D)
        qr = W.wq_kv_append_rotary(q, k, v, pos, cs, slots, kc, ks, vc, vs, interleaved=inter)
        out, lse = W.wq_kv4_attention(qr, kc, ks, vc, vs, table, cu, kv, max_q=max(new), return_lse=True)
        yield q, k, v, pos, table, cu, kv, cs, (kc, ks, vc, vs), qr, out, lse
        assert state[1].item() == 0
        ctx, cursor = kv, state[:1].clone()


@pytest.mark.parametrize("rot,inter", [(64, False), (32, True)])
def test_serving_steps(W, rot, inter):
    """Every step against the oracle on the cache as it then is, and the cache bit for bit against the
    keys and values that went in."""
    banner("kv4: prompts and decode steps together", rot, inter)
    steps = [[37, 5, 0, 90], [1, 1, 30, 1], [1, 1, 1, 1], [2, 1, 3, 1]] + [[1, 1, 1, 1]] * 6
    H, P, D = 2, 16, 64
    keys, vals = [[] for _ in steps[0]], [[] for _ in steps[0]]
    for q, k, v, pos, table, cu, kv, cs, cache, qr, out, lse in _serve(W, steps, H, 2, D, P, 8, 0, rot, inter):
        cun, kvn, posn, csn = _np(cu), _np(kv), _np(pos), host_f32(cs)
        host = [host_u8(c) for c in cache]
        q64 = qr.float().cpu().numpy().astype(np.float64)
        want = O4.rotate(q.float().cpu().numpy(), posn, csn, inter)
        assert (np.abs(q64 - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -19).all()     # |q| is below 8: fp32 roundings below 2^-20
        ref, rl, weight, spread = O4.attention(q64, cun, kvn, *host, _np(table), D ** -0.5)
        tol, tol_lse = _bounds(ref, weight, spread, int(kvn.max()), D)
        assert (np.abs(bf16_decode(host_bits16(out)) - ref) <= tol).all()
        assert (np.abs(host_f32(lse) - rl) <= tol_lse + 2.0 ** -22 * np.abs(rl)).all()
        kr = O4.rotate(k.float().cpu().numpy(), posn, csn, inter).astype(np.float32)
        for i in range(len(keys)):
            keys[i].extend(kr[cun[i]:cun[i + 1]])
            vals[i].extend(v[cun[i]:cun[i + 1]].float().cpu().numpy())
    for i in range(len(keys)):
        for j in range(len(keys[i])):
            pg, off = int(_np(table)[i, j // P]), j % P
            c, s = O4.quantize(keys[i][j])
            assert np.array_equal(host[0][pg, :, off], c) and np.array_equal(host[1][pg, :, :, off], s)
            c, s = O4.quantize(vals[i][j])
            assert np.array_equal(host[2][pg, :, :, off], c) and np.array_equal(host[3][pg, :, :, off], s)


@pytest.mark.parametrize("width", [6, 100])
def test_decode_step_in_a_graph(W, width):
    """One decode step captured once and replayed: every replay equals the eager step on the same state."""
    banner("kv4: graph replays of blocks, rotating append and attention", width)
    B, H, G, D, P = 5, 2, 4, 64, 16
    gen = torch.Generator("cuda").manual_seed(1)
    N = B * width
    start = torch.tensor([0, 15, 16, 40, 70], dtype=torch.int32, device="cuda")
    free = torch.randperm(N, device="cuda", generator=gen).int()
    cs = dev_f32(_angles(width * P, D))

    def fresh():
        t = _i32(np.full((B, width), -1))
        c = [torch.zeros(s, dtype=torch.uint8, device="cuda")
             for s in ((N, H, P, D // 2), (N, H, D // 32, P), (N, H, D // 2, P), (N, H, D // 32, P))]
        zero = torch.zeros(B, dtype=torch.int32, device="cuda")
        slots, _, _, kv, st = W.wq_kv_blocks(zero, start, free, t, P, int(start.sum()))
        g2 = torch.Generator("cuda").manual_seed(2)
        x = torch.randn(2, len(slots), H, D, device="cuda", generator=g2).to(torch.bfloat16)
        W.wq_kv4_append(x[0], x[1], slots, *c)
        return t, c, kv.clone(), st[:1].clone()

    ones = torch.ones(B, dtype=torch.int32, device="cuda")
    q = torch.empty(B, H * G, D, dtype=torch.bfloat16, device="cuda")
    k, v = (torch.empty(B, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def step(t, c, ctx, cur):
        slots, pos, cu, kv, st = W.wq_kv_blocks(ctx, ones, free, t, P, B, cursor=cur)
        qr = W.wq_kv_append_rotary(q, k, v, pos, cs, slots, *c)
        out = W.wq_kv4_attention(qr, *c, t, cu, kv, max_q=1)
        ctx.copy_(kv)
        cur.copy_(st[:1])
        return out

    def inputs(i):
        gi = torch.Generator("cuda").manual_seed(100 + i)
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, device="cuda", generator=gi))

    eager = fresh()
    want = []
    for i in range(5):
        inputs(i)
        want.append((step(*eager).clone(), eager[2].clone()))
    state = fresh()
    keep = [state[0].clone(), [c.clone() for c in state[1]], state[2].clone(), state[3].clone()]
    inputs(0)
    step(*state)                                           # warm
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*state)
    state[0].copy_(keep[0])
    for c, h in zip(state[1], keep[1]):
        c.copy_(h)
    state[2].copy_(keep[2])
    state[3].copy_(keep[3])
    other = fresh()
    for i in range(5):
        inputs(i)
        step(*other)                                       # eager work between the replays
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i][0]) and torch.equal(state[2], want[i][1]), f"replay {i}"
    for a, b in zip(state[1], eager[1]):
        assert torch.equal(a, b)


@pytest.mark.parametrize("ql", [[1, 1, 5], [1, 90, 3]])
def test_side_stream_and_repeat(W, ql):
    """Launches follow the current stream, and calls on two streams at once do not disturb each other."""
    banner("kv4: side streams", ql)
    q, cu, kv, cache, table = _problem(13, 8, 2, 128, 64, ql, [900, 4000, 300])
    args = (dev_bf16(bf16_round(q)), *[dev_u8(c) for c in cache], _i32(table), _i32(cu), _i32(kv))
    ref = W.wq_kv4_attention(*args)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in streams:
        with torch.cuda.stream(s):
            W.wq_util_spin(100000)
            outs.append([W.wq_kv4_attention(*args) for _ in range(4)])
    for s, o in zip(streams, outs):
        s.synchronize()
        assert all(torch.equal(x, ref) for x in o)


def test_workspace_of_the_caller(W):
    """A workspace of the caller, full of NaN: the same bits."""
    banner("kv4: workspace of the caller")
    for ql in ([1, 1, 2], [1, 90, 3]):
        q, cu, kv, cache, table = _problem(21, 8, 2, 128, 64, ql, [900, 4000, 300])
        args = (dev_bf16(bf16_round(q)), *[dev_u8(c) for c in cache], _i32(table), _i32(cu), _i32(kv))
        n = W.wq_kv4_attention_workspace_size(3, q.shape[0], max(ql), 8, 2, 128, 64, table.shape[1])
        ws = torch.full((max(n, 16) + 64,), 0xFF, dtype=torch.uint8, device="cuda")
        a = W.wq_kv4_attention(*args, max_q=max(ql))
        b = W.wq_kv4_attention(*args, max_q=max(ql), workspace=ws)
        assert torch.equal(a, b) and (ws[n:] == 0xFF).all()


def test_calls_through_ctypes(W, monkeypatch):
    """The same bits by the calls that go through ctypes (which those that the module of compiled calls
    refuses do) as by the compiled ones; numbers of other types go that way by themselves."""
    banner("kv4: compiled calls and ctypes")
    g = np.random.default_rng(22)
    Hq, H, D, P, T = 8, 2, 64, 16, 40
    slots, N = _slots(g, [5], [T], P)
    q, k, v = (dev_bf16(bf16_round(g.standard_normal((T, h, D)))) for h in (Hq, H, H))
    pos, cs, start = _i32(5 + np.arange(T)), dev_f32(_angles(100, D)), [_cache4(g, N, H, P, D), _cache(g, N, H, P, D)]
    args = (_i32([slots[::P] // P]), _i32([0, T]), _i32([T]))

    def everything(window=np.int64(9)):
        out = []
        for c in start:
            dev = [dev_u8(a) for a in c]
            out += [W.wq_kv_append_rotary(q, k, v, pos, cs, _i64(slots), *dev, interleaved=True), *dev]
        dev = [dev_u8(a) for a in start[0]]
        assert W.wq_kv4_append(k, v, _i64(slots), *dev) is None
        out += dev
        out += W.wq_kv4_attention(q, *dev, *args, return_lse=True)
        out.append(W.wq_kv4_attention(q, *dev, *args, window=window, softcap=20, sm_scale=1))
        mine = torch.empty_like(q)
        assert W.wq_kv4_attention(q, *dev, *args, window=9, softcap=20.0, sm_scale=1.0, out=mine) is mine
        return out + [mine]

    a = everything()
    took = []
    for name in ("kv4_append", "kv_append_rotary", "kv4_attention"):
        monkeypatch.setattr(W._calls, name, lambda *x, name=name: took.append(name) or NotImplemented)
    b = everything()
    assert len(took) == 6 and len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))
    assert torch.equal(a[-1], a[-2])


@pytest.mark.parametrize("ql", [[1, 1, 5], [40, 3, 90]])
def test_attention_nan_queries_and_keys(W, ql):
    """A query that is NaN or infinite makes its own row NaN and no other; a key with the NaN scale the rows that see it."""
    banner("kv4 attention: NaN queries and keys", ql)
    q, cu, kv, cache, table = _problem(23, 8, 2, 64, 16, ql, [300, 70, 200])
    args = (_i32(table), _i32(cu), _i32(kv))
    clean = dev_bf16(bf16_round(q))
    want = W.wq_kv4_attention(clean, *[dev_u8(c) for c in cache], *args)
    x = clean.clone()
    rows = [(0, 3), (q.shape[0] - 1, 0)]
    for t, h in rows:
        x[t, h, 5] = float("nan")
    got = W.wq_kv4_attention(x, *[dev_u8(c) for c in cache], *args)
    for t, h in rows:
        assert torch.isnan(got[t, h]).all()
        got[t, h] = want[t, h]
    assert torch.equal(got, want)
    bad = [c.copy() for c in cache]                        # the last key of request 2: its last row sees it alone
    bad[1][table[2, 199 // 16], 0, 1, 199 % 16] = 255
    got = W.wq_kv4_attention(clean, *[dev_u8(c) for c in bad], *args)
    assert torch.equal(got[:-1], want[:-1]) and torch.equal(got[-1, 4:], want[-1, 4:])


def test_append_rotary_on_a_side_stream_and_in_a_graph(W):
    """Launches follow the current stream; replays rotate in place once each, as eager calls do."""
    banner("kv append rotary: side stream, graph in place")
    g = np.random.default_rng(24)
    Hq, H, D, P, T = 4, 2, 64, 16, 33
    slots, N = _slots(g, [3], [T], P)
    q, k, v = (dev_bf16(bf16_round(g.standard_normal((T, h, D)))) for h in (Hq, H, H))
    pos, cs, sl = _i32(3 + np.arange(T)), dev_f32(_angles(60, D)), _i64(slots)
    for c in (_cache4(g, N, H, P, D), _cache(g, N, H, P, D)):
        eager, side, graphed = ([dev_u8(a) for a in c] for _ in range(3))
        want = [q.clone()]
        for _ in range(4):
            want.append(W.wq_kv_append_rotary(want[-1], k, v, pos, cs, sl, *eager).clone())
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            W.wq_util_spin(100000)
            out = W.wq_kv_append_rotary(q, k, v, pos, cs, sl, *side)
        s.synchronize()
        assert torch.equal(out, want[1]) and all(torch.equal(a, b) for a, b in zip(side, eager))
        x = q.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            W.wq_kv_append_rotary(x, k, v, pos, cs, sl, *graphed, q_out=x)
        for i in range(4):
            graph.replay()
            torch.cuda.synchronize()
            W.wq_kv_append_rotary(q, k, v, pos, cs, sl, *side)          # eager work between the replays
            torch.cuda.synchronize()
            assert torch.equal(x, want[i + 1]), f"replay {i}"
        assert all(torch.equal(a, b) for a, b in zip(graphed, eager))


def test_append_rotary_in_place_once_where_an_earlier_call_failed(W):
    """An error that another HIP call left is reported by the next launch's check; the call is not
    made a second time, which would turn queries in place twice."""
    rng = np.random.default_rng(77)
    tokens, hq, hk, d = 5, 4, 2, 64
    q, k, v = (torch.from_numpy(rng.standard_normal((tokens, h, d)).astype(np.float32)).to("cuda").bfloat16() for h in (hq, hk, hk))
    positions = torch.arange(tokens, dtype=torch.int32, device="cuda")
    angle = torch.arange(8, device="cuda")[:, None] * (0.3 / torch.arange(1, d // 2 + 1, device="cuda"))[None]
    cos_sin = torch.cat([angle.cos(), angle.sin()], 1).contiguous()
    slots = torch.arange(tokens, dtype=torch.int64, device="cuda")

    def cache():
        return [torch.zeros(s, dtype=torch.uint8, device="cuda") for s in ((1, hk, 16, d // 2), (1, hk, d // 32, 16), (1, hk, d // 2, 16), (1, hk, d // 32, 16))]

    want_cache, got_cache = cache(), cache()
    want = W.wq_kv_append_rotary(q, k, v, positions, cos_sin, slots, *want_cache)
    torch.cuda.synchronize()
    here = torch.cuda.current_device()
    assert W.lib.hipSetDevice(100000) != 0      # no such device
    try:
        W.wq_kv_append_rotary(q, k, v, positions, cos_sin, slots, *got_cache, q_out=q)
    except W.WQError as e:
        assert e.status == W.WQ_EHIP and "wq_kv_append_rotary" in str(e)
    torch.cuda.set_device(here)
    torch.cuda.synchronize()
    assert torch.equal(q, want)
    assert all(torch.equal(a, b) for a, b in zip(got_cache, want_cache))
