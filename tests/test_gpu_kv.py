"""GPU parity of the 8-bit key/value cache (block tables, append, attention)
with the oracle: tables, slots, codes and scales bit for bit, attention within
a bound on its roundings (`_bounds`)."""
import numpy as np
import pytest
import torch

from oracle import kv as OK
from oracle.formats import bf16_decode, bf16_round
from tests.gpu_helpers import banner, dev_bf16, dev_f32, dev_u8, host_bits16, host_f32, host_u8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def W():
    import weight_only_quantized_quant_amd as W
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return W


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).cuda()


def _i64(a):
    return torch.from_numpy(np.ascontiguousarray(a).astype(np.int64)).cuda()


def _np(t):
    return t.detach().cpu().numpy().astype(np.int64)


# ---------------------------------------------------------------------------
# block tables
# ---------------------------------------------------------------------------
def _check_blocks(W, ctx, new, free, cursor, page, table, tokens):
    t = _i32(table)
    got = W.wq_kv_blocks(_i32(ctx), _i32(new), _i32(free), t, page, tokens,
                         cursor=None if cursor is None else _i32([cursor]))
    want = OK.blocks(ctx, new, free, cursor or 0, page, table, tokens)
    for name, g, w in zip(("table", "slots", "positions", "cu", "kv", "state"), (t,) + tuple(got), want):
        assert np.array_equal(_np(g), w), name
    return got


@pytest.mark.parametrize("B,new_hi,page,spare,cursor", [
    (1, 1, 16, 0, None), (1, 5000, 16, 3, 0), (7, 700, 32, 0, 5), (256, 1, 64, 0, 0), (257, 3, 128, 500, 17),
    (1000, 40, 16, 0, 0), (3, 0, 64, 10, 0)])
def test_blocks(W, B, new_hi, page, spare, cursor):
    banner("kv blocks", B, new_hi, page, spare, cursor)
    g = np.random.default_rng(B + new_hi)
    ctx, new = g.integers(0, 500, B), g.integers(0, new_hi + 1, B)
    held, total = -(-ctx // page), -(-(ctx + new) // page)
    width = int(total.max()) + 2
    ids = g.permutation(int(total.sum()) + 40)
    table = np.full((B, width), -1)
    at = 0
    for i in range(B):
        table[i, :held[i]] = ids[at:at + held[i]]
        at += held[i]
    _check_blocks(W, ctx, new, np.concatenate([np.full(cursor or 0, -7), ids[at:]]), cursor, page, table,
                  int(new.sum()) + spare)


def test_blocks_refusals_on_the_device(W):
    """The list runs out, a row is too narrow, the token rows end early, negative lengths and page ids."""
    banner("kv blocks: shortage, narrow rows, few token rows, negative values")
    table = np.full((6, 3), -1)
    table[4, 0] = 77
    ctx, new = [0, 0, 0, -5, 10, 0], [20, 100, 30, -3, 2, 1]
    for tokens in (200, 160, 60, 5, 0):
        for n in (6, 5, 4, 2, 0):
            _check_blocks(W, ctx, new, np.arange(10, 10 + n), 0, 16, table, tokens)
            _check_blocks(W, ctx, new, np.arange(10, 10 + n), 2, 16, table, tokens)
    table[4, 0] = -1                                       # a page that is not there: no slot
    _check_blocks(W, ctx, new, np.arange(10), 0, 16, table, 200)
    _check_blocks(W, [2 ** 31 - 3, 0], [5, 4], np.arange(10), 0, 128, np.full((2, 3), -1), 20)


def test_blocks_empty(W):
    banner("kv blocks: no request, no token row, no free page")
    e = np.zeros(0, np.int64)
    _check_blocks(W, e, e, e, None, 16, np.zeros((0, 4), np.int64), 5)
    _check_blocks(W, e, e, e, None, 16, np.zeros((0, 4), np.int64), 0)
    _check_blocks(W, [3], [0], e, None, 16, [[4]], 0)


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
def _cache(g, N, H, P, D):
    """Random finite codes and scales around 1."""
    def codes(*s):
        c = g.integers(0, 256, s).astype(np.uint8)
        return np.where((c & 0x7F) == 0x7F, 0, c).astype(np.uint8)
    return codes(N, H, P, D), g.integers(120, 131, (N, H)).astype(np.uint8), codes(N, H, D, P), \
        g.integers(120, 131, (N, H)).astype(np.uint8)


def _check_append(W, k, v, slots, cache, bf16):
    dev = [dev_u8(c) for c in cache]
    if bf16:
        kb, vb = bf16_round(k), bf16_round(v)
        k, v = bf16_decode(kb).astype(np.float32), bf16_decode(vb).astype(np.float32)
        kd, vd = dev_bf16(kb), dev_bf16(vb)
    else:
        kd, vd = dev_f32(k), dev_f32(v)
    W.wq_kv_append(kd, vd, _i64(slots), *dev)
    kc, ks = OK.append(k, slots, cache[0], cache[1], False)
    vc, vs = OK.append(v, slots, cache[2], cache[3], True)
    for name, d, w in zip(("keys", "key scales", "values", "value scales"), dev, (kc, ks, vc, vs)):
        assert np.array_equal(host_u8(d), w), name


def _slots(g, ctx, new, page, spare=0):
    """Slots of requests with ctx tokens and new ones more, on random pages."""
    total = [-(-(c + n) // page) for c, n in zip(ctx, new)]
    ids = g.permutation(sum(total) + 3)
    out, at = [], 0
    for c, n, t in zip(ctx, new, total):
        pos = c + np.arange(n)
        out.append(ids[at + pos // page] * page + pos % page)
        at += t
    return np.concatenate(out + [np.full(spare, -1)]).astype(np.int64), len(ids)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("H,D,page,ctx,new", [
    (1, 64, 16, [0], [1]),
    (8, 128, 64, list(range(0, 640, 10)), [1] * 64),       # a decode step
    (2, 128, 16, [3, 0, 16, 31], [40, 16, 1, 2]),
    (3, 64, 32, [5, 0, 0], [100, 0, 333]),
    (1, 128, 128, [100, 1], [300, 126]),                   # runs longer than one wave
    (5, 128, 64, [63, 1], [700, 62]),
    (2, 64, 128, [7], [1500]),
])
def test_append(W, bf16, H, D, page, ctx, new):
    banner("kv append", bf16, H, D, page, ctx[:4], new[:4])
    g = np.random.default_rng(H * D + page + len(ctx))
    slots, N = _slots(g, ctx, new, page, spare=2)
    T = len(slots)
    # magnitudes from far below the pages' scales to far above: some runs move the codes before them
    amp = np.exp2(g.integers(-8, 9, (T, H, 1)))
    k, v = ((g.standard_normal((T, H, D)) * amp).astype(np.float32) for _ in range(2))
    _check_append(W, k, v, slots, _cache(g, N, H, page, D), bf16)


def test_append_many_requests_in_steps(W):
    """Enough tokens that one workgroup looks at several, in the middle of pages."""
    banner("kv append: 3000 requests x 1 token, 2 heads, pages of 16")
    g = np.random.default_rng(2)
    slots, N = _slots(g, g.integers(0, 40, 3000), [1] * 3000, 16)
    k, v = (g.standard_normal((3000, 2, 64)).astype(np.float32) for _ in range(2))
    _check_append(W, k, v, slots, _cache(g, N, 2, 16, 64), True)


@pytest.mark.parametrize("values", [1, 50])
def test_append_growing_scales(W, values):
    """Single tokens whose scale passes their page's, in every place of the page, and runs beside them."""
    banner("kv append: growing scales", values)
    g = np.random.default_rng(6)
    H, D, P = 2, 128, 32
    ctx = list(range(0, 64)) + [7, 40]
    new = [1] * 64 + [values, 3]
    slots, N = _slots(g, ctx, new, P)
    k, v = (g.standard_normal((len(slots), H, D)).astype(np.float32) * 2.0 ** g.integers(3, 7, (len(slots), H, 1))
            for _ in range(2))
    for bf16 in (True, False):
        _check_append(W, k, v, slots, _cache(g, N, H, P, D), bf16)


def test_append_special_values(W):
    banner("kv append: zeros, NaN, infinities, extremes, slots outside the cache")
    g = np.random.default_rng(3)
    H, D, P = 1, 64, 16
    k = g.standard_normal((12, H, D)).astype(np.float32)
    k[0] = 0.0
    k[1] = -0.0
    k[2, 0, :4] = [np.nan, -np.nan, np.inf, -np.inf]
    k[3] = np.nan
    k[4] = np.inf
    k[5] *= 3e38
    k[6] *= 1e-38
    k[7] *= 2.0 ** -140                                    # fp32 subnormals
    v = k[::-1].copy()
    slots = np.array([0, 17, 2 * P + 15, 3 * P, 4 * P, 5 * P, 6 * P, 7 * P + 3, -1, 12 * P, 1 << 40, 11 * P + 15])
    k = np.clip(k, -3.38e38, 3.38e38, where=np.isfinite(k), out=k)   # bf16 would round above this to infinity
    for bf16 in (True, False):
        _check_append(W, k, v, slots, _cache(g, 12, H, P, D), bf16)


def test_append_strided_rows(W):
    """Keys and values as slices of one projection's rows."""
    banner("kv append: strided keys and values")
    g = np.random.default_rng(4)
    H, D, P, T = 3, 64, 16, 50
    slots, N = _slots(g, [5], [T], P)
    bits = bf16_round(g.standard_normal((T, 5 * H * D)))
    fused = dev_bf16(bits)
    row = H * D
    k, v = (fused[:, a:a + row].view(T, H, D) for a in (3 * row, row))
    cache = _cache(g, N, H, P, D)
    dev = [dev_u8(c) for c in cache]
    W.wq_kv_append(k, v, _i64(slots), *dev)
    x = bf16_decode(bits).astype(np.float32)
    for d, (w, s), i in ((dev, OK.append(x[:, 3 * row:4 * row].reshape(T, H, D), slots, cache[0], cache[1], False), 0),
                         (dev, OK.append(x[:, row:2 * row].reshape(T, H, D), slots, cache[2], cache[3], True), 2)):
        assert np.array_equal(host_u8(d[i]), w) and np.array_equal(host_u8(d[i + 1]), s)


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def _bounds(ref, weight, spread, seen, D):
    """What roundings may change.  Output: half a bf16 step (2^-8 relative) of the result, and of
    every probability before the second product (2^-8 of sum w |v|).  A score is a sum of D
    products and a few scalings in fp32: off by at most e = (D + 16) 2^-24 max sum |q k|, which
    moves a probability and the sum by the factor exp(2 e); the sums over `seen` tokens add at most
    seen 2^-23 relative, the exponentials and the division 2^-20."""
    e = (D + 16) * 2.0 ** -24 * spread
    rel = np.expm1(2 * e) + (seen + 8) * 2.0 ** -23 + 2.0 ** -20
    tol_out = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + rel)[..., None] * 1.01 * weight + 1e-30
    return tol_out, e + (seen + 8) * 2.0 ** -23 + 2.0 ** -20


def _check_attention(W, q, cu, kv, cache, table, rows=None, poison=True, **kw):
    """q fp64 [T, Hq, D].  `poison`: bytes and scales the call must not use become NaN."""
    N, H, P, D = cache[0].shape
    T = q.shape[0]
    bits = bf16_round(q)
    q64 = bf16_decode(bits)
    opts = {"sm_scale": D ** -0.5, "softcap": 0.0, "window": 0}
    opts.update({k: kw[k] for k in opts if k in kw})
    ref, lse, weight, spread = OK.attention(q64, cu, kv, *cache, table, **opts)
    cache = [c.copy() for c in cache]
    if poison:
        used = np.zeros((N, P), bool)
        for i, m in enumerate(kv):
            for j in range(0, min(int(m), table.shape[1] * P)):
                pg = table[i][j // P]
                if 0 <= pg < N:
                    used[pg, j % P] = True
        idle = ~used.any(1)
        cache[1][idle], cache[3][idle] = 255, 255
        cache[0][np.nonzero(~used)[0], :, np.nonzero(~used)[1]] = 0x7F
        cache[2].transpose(0, 3, 1, 2)[~used] = 0xFF
    out = torch.full((T, q.shape[1], D), 7.0, dtype=torch.bfloat16, device="cuda")
    got, glse = W.wq_kv_attention(dev_bf16(bits), *[dev_u8(c) for c in cache], _i32(table), _i32(cu), _i32(kv),
                                  out=out, return_lse=True, **kw)
    torch.cuda.synchronize()
    y, l = bf16_decode(host_bits16(got)), host_f32(glse).astype(np.float64)
    real = ~np.isnan(ref[:, 0, 0])
    assert (y[~real] == 7.0).all(), "rows behind the last request changed"
    seen = max(1, min(int(max(kv, default=1)), table.shape[1] * P))
    tol, tol_lse = _bounds(ref[real], weight[real], spread[real], seen, D)
    assert np.isfinite(y[real]).all()
    worst = (np.abs(y[real] - ref[real]) / tol).max(initial=0.0)
    assert worst <= 1.0, f"output: error / bound = {worst:.3f}"
    none = np.isneginf(lse[real])
    assert np.array_equal(none, np.isneginf(l[real]))
    with np.errstate(invalid="ignore"):
        d = np.where(none, 0.0, np.abs(l[real] - lse[real]) / (tol_lse + 2.0 ** -22 * np.abs(lse[real])))
    assert d.max(initial=0.0) <= 1.0, f"lse: error / bound = {d.max():.3f}"
    return got


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
    return q, np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int64), list(kv_lens), _cache(g, N, H, P, D), table


SHAPES = [
    # Hq, H, D, page, query lengths, cache lengths
    (1, 1, 64, 16, [1], [1]),
    (4, 4, 128, 16, [1, 1, 1], [5, 64, 129]),              # one query head a key head
    (32, 8, 128, 64, [1] * 5, [1, 63, 64, 65, 700]),
    (16, 2, 64, 128, [1, 1], [1000, 17]),
    (24, 1, 128, 32, [1, 1], [300, 2]),                    # more query heads than a 16-row tile
    (5, 1, 128, 32, [4, 1, 3, 0], [200, 50, 3, 40]),       # rows that do not fill a tile, an empty request
    (8, 2, 64, 16, [130, 1, 33], [130, 77, 300]),          # prompt, decode and chunk in one batch
    (8, 2, 128, 64, [200], [520]),
    (4, 4, 128, 128, [300], [300]),
    (6, 2, 64, 64, [129, 70], [129, 1000]),
    (128, 1, 64, 64, [1, 1, 2], [700, 90, 64]),            # more rows than a decode tile takes, for one token
    (66, 2, 128, 16, [1, 1], [40, 1500]),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}x{s[1]}x{s[2]}p{s[3]}")
@pytest.mark.parametrize("hint", [0, 1, "max"])
def test_attention(W, shape, hint):
    Hq, H, D, P, ql, kl = shape
    banner("kv attention", shape, hint)
    q, cu, kv, cache, table = _problem(1, Hq, H, D, P, ql, kl, spare_rows=3)
    _check_attention(W, q, cu, kv, cache, table, max_q=max(ql) if hint == "max" else hint)


@pytest.mark.parametrize("shape", SHAPES[1:], ids=lambda s: f"{s[0]}x{s[1]}x{s[2]}p{s[3]}")
@pytest.mark.parametrize("softcap,window", [(0.0, 1), (0.0, 50), (5.0, 0), (20.0, 64), (0.0, 100000)])
def test_attention_window_and_cap(W, shape, softcap, window):
    Hq, H, D, P, ql, kl = shape
    banner("kv attention window / cap", shape, softcap, window)
    q, cu, kv, cache, table = _problem(2, Hq, H, D, P, ql, kl)
    _check_attention(W, q, cu, kv, cache, table, softcap=softcap, window=window, sm_scale=0.02)


@pytest.mark.parametrize("ql", [[1, 1, 1, 1], [40, 3, 150, 1]])
def test_attention_rows_that_see_nothing(W, ql):
    """No cache at all, fewer tokens than queries, a window on pages that are not there."""
    banner("kv attention: rows without a token", ql)
    kl = [0, 2, 20, 33]
    q, cu, kv, cache, table = _problem(3, 8, 2, 64, 16, ql, kl)
    _check_attention(W, q, cu, kv, cache, table)
    table[3, 2] = -1
    table[2, 0] = len(cache[1])
    _check_attention(W, q, cu, kv, cache, table)
    _check_attention(W, q, cu, kv, cache, table, window=1)


@pytest.mark.parametrize("ql", [[1, 1], [90, 2]])
def test_attention_pages_that_are_not_there(W, ql):
    banner("kv attention: page ids outside the cache", ql)
    q, cu, kv, cache, table = _problem(4, 4, 2, 128, 16, ql, [300, 170])
    table[0, [0, 3, 4, 9]] = [-1, 1 << 30, -(1 << 31), len(cache[1])]
    table[1, 10] = -5
    _check_attention(W, q, cu, kv, cache, table)


def test_attention_lengths_outside_the_contract(W):
    """Lengths past the table, negative ones and row ranges past the arrays are clamped."""
    banner("kv attention: lengths and ranges that do not fit")
    q, cu, kv, cache, table = _problem(5, 4, 2, 64, 16, [2, 3, 1, 2], [40, 20, 9, 30], spare_cols=0)
    got = _check_attention(W, q, cu, [1000, -7, 9, 30], cache, table, poison=False)
    assert got.shape[0] == 8
    for bad in ([0, 2, 5, 4, 100], [-3, 2, 5, 6, 8], [0, 2 ** 31 - 1, 5, 6, 8], [5, 4, 3, 2, 1]):
        for hint in (0, 1):
            out = W.wq_kv_attention(dev_bf16(bf16_round(q)), *[dev_u8(c) for c in cache], _i32(table), _i32(bad),
                                    _i32(kv), max_q=hint)
            torch.cuda.synchronize()
            assert out.shape == q.shape


def test_attention_shared_pages_and_scales(W):
    """Two requests on the same first pages; scales of a page and head apart by 2^40."""
    banner("kv attention: shared prefix, far scales")
    q, cu, kv, cache, table = _problem(6, 8, 2, 128, 32, [1, 3, 70], [100, 130, 200])
    table[1, :3] = table[0, :3]
    table[2, :2] = table[0, :2]
    g = np.random.default_rng(6)
    cache[3][:] = g.integers(100, 141, cache[3].shape)
    cache[1][:] = g.integers(90, 121, cache[1].shape)
    _check_attention(W, q, cu, kv, cache, table, poison=False)


def test_attention_extreme_scores(W):
    """Scores of some thousands: one token takes everything, in the first or the last tile."""
    banner("kv attention: peaked scores")
    for seed in range(2):
        q, cu, kv, cache, table = _problem(7 + seed, 4, 1, 64, 16, [1, 20], [333, 500])
        q *= 40
        if seed:
            cache[1][:] = 127
        _check_attention(W, q, cu, kv, cache, table, sm_scale=1e-3)


@pytest.mark.parametrize("ql", [[1, 3, 1], [40, 1, 90]])
@pytest.mark.parametrize("softcap,sm_scale", [(2.0, 1.0), (30.0, 0.5), (1000.0, 0.05), (0.002, 0.01), (50.0, 1e-4)])
def test_attention_caps(W, ql, softcap, sm_scale):
    """Scores far above their cap and far below it, in one tile and apart."""
    banner("kv attention: caps", ql, softcap, sm_scale)
    q, cu, kv, cache, table = _problem(17, 8, 2, 64, 16, ql, [300, 70, 500])
    cache[1][:] = np.random.default_rng(17).integers(110, 128, cache[1].shape)
    cache[0][:] = np.where((cache[0] & 0x78) > 0x50, cache[0] & 0x87, cache[0])   # keys of up to 30, most below 1
    _check_attention(W, q, cu, kv, cache, table, softcap=softcap, sm_scale=sm_scale)


def test_attention_strided_queries(W):
    banner("kv attention: queries as slices of wider rows")
    q, cu, kv, cache, table = _problem(9, 8, 2, 64, 16, [1, 40, 3], [50, 40, 9])
    bits = bf16_round(q)
    wide = torch.zeros((q.shape[0], 3 * 8 * 64), dtype=torch.bfloat16, device="cuda")
    mid = wide[:, 512:1024].view(-1, 8, 64)
    mid.copy_(dev_bf16(bits))
    dev = [dev_u8(c) for c in cache]
    args = (*dev, _i32(table), _i32(cu), _i32(kv))
    a, b = W.wq_kv_attention(mid, *args), W.wq_kv_attention(dev_bf16(bits), *args)
    assert torch.equal(a, b)


def test_attention_one_long_context_beside_short_ones(W):
    banner("kv attention: 20000 tokens beside short contexts")
    q, cu, kv, cache, table = _problem(10, 4, 2, 64, 64, [1, 1, 1, 2], [20000, 3, 900, 5000])
    _check_attention(W, q, cu, kv, cache, table, poison=False)


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("H,group,most_q,D", [(8, 2, 1, 64), (8, 4, 6, 64), (5, 3, 1, 128), (16, 2, 10, 128), (3, 16, 4, 64)])
def test_attention_shares_over_requests(W, page, H, group, most_q, D):
    """Ragged batches whose tiles are cut into shares that begin and end anywhere: several requests to
    a wave, several waves to a request, requests without rows or without a cache between them."""
    banner("kv attention: shares over requests", page, H, group, most_q, D)
    g = np.random.default_rng(H + page)
    kl = np.exp(g.uniform(0, np.log(3000), 40)).astype(int)
    ql = g.integers(1, most_q + 1, 40)
    kl[[3, 17]], ql[[5, 6, 30]], kl[[9, 22]] = 0, 0, [2999, 2048]
    q, cu, kv, cache, table = _problem(14, H * group, H, D, page, ql, kl, spare_rows=2)
    for kw in ({}, {"window": 700}):
        _check_attention(W, q, cu, kv, cache, table, max_q=most_q, **kw)


@pytest.mark.parametrize("hint", [0, 1])
def test_attention_many_short_requests(W, hint):
    banner("kv attention: 900 requests of a few tokens, 16 key heads", hint)
    g = np.random.default_rng(15)
    kl, ql = g.integers(0, 130, 900), g.integers(0, 3, 900)
    q, cu, kv, cache, table = _problem(15, 16, 16, 64, 16, ql, kl)
    _check_attention(W, q, cu, kv, cache, table, max_q=2 if hint else 0)


@pytest.mark.parametrize("page", [32, 64])
def test_attention_chunk_of_a_long_prompt(W, page):
    """Few rows and many tokens: prompt tiles are split over the cache, beside short requests."""
    banner("kv attention: chunks of 40 and 90 rows on 3000 tokens", page)
    q, cu, kv, cache, table = _problem(16, 8, 2, 128, page, [40, 1, 90, 5], [3000, 700, 2500, 64])
    for kw in ({}, {"softcap": 10.0}, {"window": 1500}):
        _check_attention(W, q, cu, kv, cache, table, **kw)


def test_attention_cache_past_32_bits(W):
    """Pages whose bytes lie beyond 2^32."""
    banner("kv attention and append: a cache of 4.6 GB codes each")
    N, H, P, D = 70000, 8, 64, 128
    kc = torch.empty((N, H, P, D), dtype=torch.uint8, device="cuda")
    vc = torch.empty((N, H, D, P), dtype=torch.uint8, device="cuda")
    ks, vs = (torch.empty((N, H), dtype=torch.uint8, device="cuda") for _ in range(2))
    g = np.random.default_rng(11)
    pages = np.array([69999, 3, 65536, 40000])
    k, v = (bf16_round(g.standard_normal((200, H, D))) for _ in range(2))
    slots = np.concatenate([p * P + np.arange(P) for p in pages])[:200]
    W.wq_kv_append(dev_bf16(k), dev_bf16(v), _i64(slots), kc, ks, vc, vs)
    small = [np.zeros((4, H, P, D), np.uint8), np.zeros((4, H), np.uint8), np.zeros((4, H, D, P), np.uint8),
             np.zeros((4, H), np.uint8)]
    at = np.concatenate([i * P + np.arange(P) for i in range(4)])[:200]
    small[0], small[1] = OK.append(bf16_decode(k).astype(np.float32), at, small[0], small[1], False)
    small[2], small[3] = OK.append(bf16_decode(v).astype(np.float32), at, small[2], small[3], True)
    qb = bf16_round(g.standard_normal((3, 16, D)))
    args = (_i32([[0, 1, 2, 3]] * 2), _i32([0, 1, 3]), _i32([150, 200]))
    a = W.wq_kv_attention(dev_bf16(qb), *[dev_u8(c) for c in small], *args)
    b = W.wq_kv_attention(dev_bf16(qb), kc, ks, vc, vs, _i32([pages] * 2), *args[1:])
    assert torch.equal(a, b)
    assert np.array_equal(host_u8(kc[_i64(pages[:3])]), small[0][:3])


def test_refusals_of_the_binding(W):
    banner("kv: shapes and types the binding refuses")
    q, cu, kv, cache, table = _problem(12, 4, 2, 64, 16, [2], [20])
    x, c = dev_bf16(bf16_round(q)), [dev_u8(a) for a in cache]
    t, u, n = _i32(table), _i32(cu), _i32(kv)
    ok = lambda q=x, c=c, t=t, u=u, n=n, **kw: W.wq_kv_attention(q, *c, t, u, n, **kw)
    ok()
    for bad in (dict(q=x.float()), dict(q=x[:, :3].contiguous()), dict(q=x.transpose(0, 1)), dict(t=t.long()),
                dict(t=t[0]), dict(u=u[:1]), dict(n=n.repeat(2)), dict(n=n.cpu()), dict(c=c[:3] + [c[1].int()]),
                dict(c=[c[0], c[1], c[0], c[3]]), dict(softcap=-1.0), dict(window=-2), dict(sm_scale=0.0),
                dict(max_q=-1), dict(out=torch.empty_like(x)[:1]),
                dict(workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
                if W.wq_kv_attention_workspace_size(1, 2, 0, 4, 2, 64, 16, t.shape[1]) else dict(window=-1)):
        with pytest.raises(ValueError):
            ok(**bad)
    k = torch.zeros((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    s = _i64([0, 1])
    for bad in ((k[:, :1], k, s), (k, k.float(), s), (k.half(), k.half(), s), (k, k, s.int()), (k, k, s[:1]),
                (k.transpose(1, 2).contiguous().transpose(1, 2), k, s)):
        with pytest.raises(ValueError):
            W.wq_kv_append(*bad, *c)
    i = _i32([1, 2])
    tab = _i32(np.zeros((2, 2)))
    for bad in ((i.long(), i, i, tab, 16, 3), (i, i[:1], i, tab, 16, 3), (i, i, i, tab[:1], 16, 3),
                (i, i, i.long(), tab, 16, 3), (i, i, i, tab, 24, 3), (i, i, i, tab, 16, -1), (i, i, i, i, 16, 3)):
        with pytest.raises(ValueError):
            W.wq_kv_blocks(*bad)


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
def _serve(W, steps, H, G, D, P, width, seed):
    """Prompts, then decode steps: lengths, tables, slots and cursor stay on the device."""
    g = torch.Generator("cuda").manual_seed(seed)
    B = len(steps[0])
    N = B * width + 1
    kc = torch.full((N, H, P, D), 0x7F, dtype=torch.uint8, device="cuda")
    vc = torch.full((N, H, D, P), 0x7F, dtype=torch.uint8, device="cuda")
    ks, vs = (torch.full((N, H), 255, dtype=torch.uint8, device="cuda") for _ in range(2))
    table = _i32(np.full((B, width), -1))
    free = torch.randperm(N, device="cuda", generator=g).int()
    ctx, cursor = _i32(np.zeros(B)), _i32([0])
    for new in steps:
        T = sum(new)
        slots, pos, cu, kv, state = W.wq_kv_blocks(ctx, _i32(new), free, table, P, T, cursor=cursor)
        qkv = torch.randn(T, (H * G + 2 * H) * D, device="cuda", generator=g).to(torch.bfloat16)
        k = qkv[:, H * G * D:(H * G + H) * D].view(T, H, D)
        v = qkv[:, (H * G + H) * D:].view(T, H, D)
        W.wq_kv_append(k, v, slots, kc, ks, vc, vs)
        q = qkv[:, :H * G * D].view(T, H * G, D)
        out, lse = W.wq_kv_attention(q, kc, ks, vc, vs, table, cu, kv, max_q=max(new), return_lse=True)
        yield q, k, v, pos, table, cu, kv, (kc, ks, vc, vs), out, lse
        assert state[1].item() == 0
        ctx, cursor = kv, state[:1].clone()


def test_serving_steps(W):
    """Every step against the oracle on the cache as it then is, and the cache against the keys and
    values that went in: each within a half step of its page's scale per rounding."""
    banner("kv: prompts and decode steps together")
    steps = [[37, 5, 0, 90], [1, 1, 30, 1], [1, 1, 1, 1], [2, 1, 3, 1]] + [[1, 1, 1, 1]] * 12
    H, P, D = 2, 16, 64
    keys = [[] for _ in steps[0]]
    for q, k, v, pos, table, cu, kv, cache, out, lse in _serve(W, steps, H, 2, D, P, 8, 0):
        cun, kvn = _np(cu), _np(kv)
        host = [host_u8(c) for c in cache]
        q64 = q.float().cpu().numpy().astype(np.float64)
        ref, rl, weight, spread = OK.attention(q64, cun, kvn, *host, _np(table), D ** -0.5)
        tol, tol_lse = _bounds(ref, weight, spread, int(kvn.max()), D)
        assert (np.abs(bf16_decode(host_bits16(out)) - ref) <= tol).all()
        assert (np.abs(host_f32(lse) - rl) <= tol_lse + 2.0 ** -22 * np.abs(rl)).all()
        for i in range(len(keys)):
            keys[i].extend(k[cun[i]:cun[i + 1]].float().cpu().numpy())
        assert _np(pos).tolist() == [p for i in range(len(keys)) for p in range(kvn[i] - cun[i + 1] + cun[i], kvn[i])]
    for i, kk in enumerate(keys):
        for j, want in enumerate(kk):
            pg = int(_np(table)[i, j // P])
            unit = np.exp2(host[1][pg].astype(np.float64) - 127)[:, None]
            from oracle.formats import e4m3_decode
            got = e4m3_decode(host[0][pg, :, j % P]) * unit
            # a page's scale grows at most 16 times here, but each growth at least doubles it: the
            # rounding errors of normal codes halve with each, so 2 half steps relative, and half a
            # subnormal step of each scale up to the last one, 2^-10 (1 + 1/2 + ...) of it
            assert (np.abs(got - want) <= 2 * 2.0 ** -4 * np.abs(want) + 2 * 2.0 ** -10 * unit).all()


@pytest.mark.parametrize("width", [6, 100])                # 100: wide enough that contexts are split
def test_decode_step_in_a_graph(W, width):
    """One decode step captured once and replayed: every replay equals the eager step on the same state."""
    banner("kv: graph replays of blocks, append and attention", width)
    B, H, G, D, P = 5, 2, 4, 64, 16
    gen = torch.Generator("cuda").manual_seed(1)
    N = B * width
    start = torch.tensor([0, 15, 16, 40, 70], dtype=torch.int32, device="cuda")
    free = torch.randperm(N, device="cuda", generator=gen).int()

    def fresh():
        t = _i32(np.full((B, width), -1))
        c = [torch.zeros(s, dtype=torch.uint8, device="cuda")
             for s in ((N, H, P, D), (N, H), (N, H, D, P), (N, H))]
        zero = torch.zeros(B, dtype=torch.int32, device="cuda")
        slots, _, _, kv, st = W.wq_kv_blocks(zero, start, free, t, P, int(start.sum()))
        g2 = torch.Generator("cuda").manual_seed(2)
        x = torch.randn(2, len(slots), H, D, device="cuda", generator=g2).to(torch.bfloat16)
        W.wq_kv_append(x[0], x[1], slots, *c)
        return t, c, kv.clone(), st[:1].clone()

    ones = torch.ones(B, dtype=torch.int32, device="cuda")
    q = torch.empty(B, H * G, D, dtype=torch.bfloat16, device="cuda")
    k, v = (torch.empty(B, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def step(t, c, ctx, cur):
        slots, _, cu, kv, st = W.wq_kv_blocks(ctx, ones, free, t, P, B, cursor=cur)
        W.wq_kv_append(k, v, slots, *c)
        out = W.wq_kv_attention(q, *c, t, cu, kv, max_q=1)
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


def test_side_stream_and_repeat(W):
    """Launches follow the current stream, and calls on two streams at once do not disturb each other."""
    banner("kv: side streams")
    q, cu, kv, cache, table = _problem(13, 8, 2, 128, 64, [1, 1, 5], [900, 4000, 300])
    args = (dev_bf16(bf16_round(q)), *[dev_u8(c) for c in cache], _i32(table), _i32(cu), _i32(kv))
    ref = W.wq_kv_attention(*args)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in streams:
        with torch.cuda.stream(s):
            W.wq_util_spin(100000)
            outs.append([W.wq_kv_attention(*args) for _ in range(4)])
    for s, o in zip(streams, outs):
        s.synchronize()
        assert all(torch.equal(x, ref) for x in o)
