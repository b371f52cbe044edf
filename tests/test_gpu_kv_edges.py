"""The 8-bit key/value cache where it can go wrong unseen: softmaxes whose
weights are spread over many tokens, small ratios of scale and cap, bytes that
no row or not every row sees, NaN and infinite values, caller-owned workspaces."""
import numpy as np
import pytest
import torch

from oracle import kv as OK
from oracle.e4m3 import e4m3_from_f32
from oracle.formats import bf16_decode, bf16_round
from tests.gpu_helpers import banner, dev_bf16, dev_u8, host_bits16, host_f32
from tests.test_gpu_kv import W, _bounds, _i32, _problem  # noqa: F401 (W is a fixture)

pytestmark = pytest.mark.gpu


def _spread_problem(seed, Hq, H, D, P, q_lens, kv_lens, spare_cols=1):
    """Scores of a standard deviation of 1.5 at the default scale: keys and values quantized from
    normal numbers, page scales up to 2^6 apart."""
    q, cu, kv, cache, table = _problem(seed, Hq, H, D, P, q_lens, kv_lens, spare_cols=spare_cols)
    g = np.random.default_rng(seed + 1000)
    N = len(cache[1])
    out = []
    for shape in ((N, H, P, D), (N, H, D, P)):
        c = g.integers(124, 131, (N, H))
        x = g.standard_normal(shape)
        out += [e4m3_from_f32(np.ldexp(x, 127 - c[..., None, None]).astype(np.float32)), c.astype(np.uint8)]
    return 3 * q, cu, kv, out, table


def _attend(W, q, cu, kv, cache, table, **kw):
    """Bits of out and of lse."""
    out, lse = W.wq_kv_attention(dev_bf16(bf16_round(q)), *[dev_u8(c) for c in cache], _i32(table), _i32(cu), _i32(kv),
                                 return_lse=True, **kw)
    torch.cuda.synchronize()
    return host_bits16(out), host_f32(lse).view(np.uint32)


def _compare(bits, lse_bits, q, cu, kv, cache, table, sm_scale=None, softcap=0.0, window=0):
    """Within the bound of the roundings; a capped score is off by softcap * 2^-22 more."""
    D = q.shape[2]
    ref, rl, weight, spread = OK.attention(bf16_decode(bf16_round(q)), cu, kv, *cache, table,
                                           D ** -0.5 if sm_scale is None else sm_scale, softcap, window)
    seen = int(max(kv))
    e = softcap * 2.0 ** -22
    tol, tol_lse = _bounds(ref, weight, spread + e / ((D + 16) * 2.0 ** -24), seen, D)
    y, l = bf16_decode(bits), lse_bits.view(np.float32).astype(np.float64)
    some = ~np.isneginf(rl)                                   # rows that see a token
    assert np.array_equal(np.isfinite(l), some) and np.isneginf(l[~some]).all() and (y[~some] == 0).all()
    assert np.isfinite(y).all()
    worst = (np.abs(y - ref) / tol).max()
    assert worst <= 1.0, f"output: error / bound = {worst:.3f}"
    worst = (np.abs(l[some] - rl[some]) / (tol_lse[some] + 2.0 ** -22 * np.abs(rl[some]))).max()
    assert worst <= 1.0, f"lse: error / bound = {worst:.3f}"


# ---------------------------------------------------------------------------
# capped scores
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("ql", [[1, 3], [70, 1]])
@pytest.mark.parametrize("log_k", [10, 20, 32, 66, 90])
@pytest.mark.parametrize("log_x", [-8, -7, -4])               # below a quarter of the cap, about it, above it
def test_attention_cap_of_a_small_scale(W, ql, log_k, log_x):
    """sm_scale / softcap far below 1, beside keys whose scales make up for it: dots of 2^log_k."""
    banner("kv attention: scale / cap of 2^-", log_k, log_x, ql)
    q, cu, kv, cache, table = _spread_problem(31, 8, 2, 64, 16, ql, [300, 70])
    g = np.random.default_rng(31)
    q = np.abs(q) / 3                                         # dots of one sign: what the cap takes away adds up
    cache[0] = g.integers(0x28, 0x40, cache[0].shape).astype(np.uint8)
    cache[1][:] = 127 + log_k + log_x
    for softcap in (1.0, 300.0):
        kw = {"softcap": softcap, "sm_scale": softcap * 2.0 ** -log_k}
        _compare(*_attend(W, q, cu, kv, cache, table, **kw), q, cu, kv, cache, table, **kw)


# ---------------------------------------------------------------------------
# bytes that no row sees
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("Hq,H,D,P,ql", [(8, 2, 128, 64, [1, 1, 1]), (4, 4, 64, 16, [1, 3, 2]), (8, 2, 64, 128, [5, 1, 4]),
                                         (8, 2, 128, 64, [90, 1, 40]), (4, 2, 64, 32, [130, 3, 70])])
@pytest.mark.parametrize("softcap", [0.0, 50.0])
def test_attention_does_not_depend_on_bytes_no_row_sees(W, Hq, H, D, P, ql, softcap):
    """Stale keys and values behind a request's length, before its window and in page 0, which is
    read in place of a missing page: large ones give the bits that zeros give."""
    banner("kv attention: unseen bytes", Hq, H, D, P, ql, softcap)
    kl, window = [331, 90, 301], 150
    q, cu, kv, cache, table = _spread_problem(32, Hq, H, D, P, ql, kl)
    table = np.where(table >= 0, table + 1, -1)               # page 0 is nobody's
    cache = [np.concatenate([c[:1], c]) for c in cache]
    table[2, 300 // P - 1] = -1
    for win in (0, window):
        seen = np.zeros((len(cache[1]), P), bool)
        for i, m in enumerate(kl):
            for j in range(max(0, m - ql[i] - win + 1) if win else 0, m):
                if table[i, j // P] >= 0:
                    seen[table[i, j // P], j % P] = True
        got = []
        for code in (0x00, 0x7E, 0xFE):
            c = [x.copy() for x in cache]
            c[0][np.nonzero(~seen)[0], :, np.nonzero(~seen)[1]] = code
            c[2].transpose(0, 3, 1, 2)[~seen] = code
            got.append(_attend(W, q, cu, kv, c, table, softcap=softcap, window=win))
        for name, at in (("out", 0), ("lse", 1)):
            for other in got[1:]:
                assert np.array_equal(got[0][at], other[at]), (name, win)
        # what the zeros give is right
        zeros = [x.copy() for x in cache]
        zeros[0][np.nonzero(~seen)[0], :, np.nonzero(~seen)[1]] = 0
        _compare(*got[0], q, cu, kv, zeros, table, softcap=softcap, window=win)


# ---------------------------------------------------------------------------
# NaN and infinite values
# ---------------------------------------------------------------------------
def _rows_that_see(cu, kv, i, j, window):
    """Rows of request i that see its token j."""
    n = int(cu[i + 1] - cu[i])
    pos = kv[i] - n + np.arange(n)
    return cu[i] + np.nonzero((pos >= j) & ((pos - j < window) if window else True))[0]


VALUE_SHAPES = [
    # Hq, H, D, page, query lengths, cache lengths, spare columns of the table, window
    (8, 2, 128, 64, [5, 3, 1], [200, 66, 90], 1, 0),           # a workgroup a row tile
    (4, 2, 64, 16, [7, 4, 2], [300, 129, 40], 1, 40),
    (8, 2, 128, 32, [6, 8, 2], [700, 1400, 64], 200, 0),       # shares of tiles
    (16, 2, 64, 128, [2, 7, 1], [900, 3000, 5], 100, 3),
    (8, 2, 128, 64, [130, 70, 40], [330, 70, 200], 1, 0),      # prompts
    (4, 4, 64, 16, [200, 129, 3], [200, 300, 77], 1, 0),
    (6, 2, 128, 16, [90, 50, 1], [150, 800, 9], 1, 30),
    (8, 2, 64, 128, [64, 40, 64], [3000, 2500, 64], 1, 700),   # rows split over the cache
]


@pytest.mark.parametrize("shape", VALUE_SHAPES, ids=lambda s: f"{s[0]}x{s[1]}x{s[2]}p{s[3]}w{s[7]}")
@pytest.mark.parametrize("softcap", [0.0, 20.0])
def test_attention_value_that_is_not_finite(W, shape, softcap):
    """A NaN value, or one whose scale takes it past bf16, reaches its own channel of the rows that
    see its token, and nothing else: the rest has the bits that a zero in its place gives."""
    Hq, H, D, P, ql, kl, spare, window = shape
    banner("kv attention: values that are not finite", shape, softcap)
    q, cu, kv, cache, table = _spread_problem(33, Hq, H, D, P, ql, kl, spare_cols=spare)
    G = Hq // H
    for i in range(2):
        for back in sorted({0, 1, ql[i] // 2, ql[i] - 1, min(ql[i] + 5, kl[i] - 1)}):
            j, head, ch = kl[i] - 1 - back, (i + back) % H, (37 * back + 11) % D
            page = table[i, j // P]
            for code, scale in ((0x7F, None), (0xFF, None), (0x7E, 250), (0xFA, 247)):
                c = [x.copy() for x in cache]
                if scale is not None:                          # the others of the page stay below 2^-4
                    c[3][page, head] = scale
                    c[2][page, head] &= 0x97
                c[2][page, head, ch, j % P] = 0
                want, want_lse = _attend(W, q, cu, kv, c, table, softcap=softcap, window=window)
                assert np.isfinite(bf16_decode(want)).all()
                c[2][page, head, ch, j % P] = code
                got, lse = _attend(W, q, cu, kv, c, table, softcap=softcap, window=window)
                hit = np.zeros(got.shape, bool)
                hit[_rows_that_see(cu, kv, i, j, window), head * G:(head + 1) * G, ch] = True
                y = bf16_decode(got)
                assert not np.isfinite(y[hit]).any(), (i, back, code)
                if scale is None:
                    assert np.isnan(y[hit]).all(), (i, back, code)
                assert np.array_equal(got[~hit], want[~hit]) and np.array_equal(lse, want_lse), (i, back, code)


@pytest.mark.parametrize("shape", VALUE_SHAPES, ids=lambda s: f"{s[0]}x{s[1]}x{s[2]}p{s[3]}w{s[7]}")
def test_attention_nan_keys_and_queries(W, shape):
    """A NaN key makes the rows that see it NaN, a NaN query its own row, and no others."""
    Hq, H, D, P, ql, kl, spare, window = shape
    banner("kv attention: NaN keys and queries", shape)
    q, cu, kv, cache, table = _spread_problem(34, Hq, H, D, P, ql, kl, spare_cols=spare)
    G = Hq // H
    for softcap in (0.0, 20.0):
        want, want_lse = _attend(W, q, cu, kv, cache, table, softcap=softcap, window=window)
        for i, back in ((0, ql[0] // 2), (1, 0), (1, min(ql[1] + 5, kl[1] - 1))):
            j, head = kl[i] - 1 - back, back % H
            c = [x.copy() for x in cache]
            c[0][table[i, j // P], head, j % P, 5] = 0x7F
            got, lse = _attend(W, q, cu, kv, c, table, softcap=softcap, window=window)
            hit = np.zeros(want_lse.shape, bool)
            hit[_rows_that_see(cu, kv, i, j, window), head * G:(head + 1) * G] = True
            assert np.isnan(bf16_decode(got)[hit]).all() and np.isnan(lse.view(np.float32)[hit]).all()
            assert np.isfinite(bf16_decode(got)[~hit]).all() and np.isfinite(lse.view(np.float32)[~hit]).all()
        x = q.copy()
        x[1, 1, 3] = np.nan
        got, lse = _attend(W, x, cu, kv, cache, table, softcap=softcap, window=window)
        hit = np.zeros(want_lse.shape, bool)
        hit[1, 1] = True
        assert np.isnan(bf16_decode(got)[hit]).all() and np.isnan(lse.view(np.float32)[hit]).all()
        assert np.isfinite(bf16_decode(got)[~hit]).all() and np.isfinite(lse.view(np.float32)[~hit]).all()


@pytest.mark.parametrize("ql", [[1, 2], [70, 1]])
def test_attention_largest_scale(W, ql):
    """sm_scale 2^127: a query of zeros sees all its tokens alike."""
    banner("kv attention: the largest scale", ql)
    q, cu, kv, cache, table = _spread_problem(39, 4, 2, 64, 16, ql, [200, 70])
    kw = {"sm_scale": 2.0 ** 127}
    _compare(*_attend(W, 0 * q, cu, kv, cache, table, **kw), 0 * q, cu, kv, cache, table, **kw)
    with pytest.raises(ValueError):
        W.wq_kv_attention(dev_bf16(bf16_round(q)), *[dev_u8(c) for c in cache], _i32(table), _i32(cu), _i32(kv), sm_scale=3e38)


# ---------------------------------------------------------------------------
# workspaces
# ---------------------------------------------------------------------------
def test_workspace_of_another_kind_is_refused(W):
    banner("kv attention: workspaces that are no tensors on the GPU")
    q, cu, kv, cache, table = _spread_problem(35, 8, 2, 64, 16, [1, 1], [100, 60])
    args = (dev_bf16(bf16_round(q)), *[dev_u8(c) for c in cache], _i32(table), _i32(cu), _i32(kv))
    for bad in (1 << 20, bytearray(1 << 20), np.zeros(1 << 20, np.uint8), torch.zeros(1 << 20, dtype=torch.uint8),
                torch.zeros((1 << 10, 2), dtype=torch.uint8, device="cuda")[:, :1]):
        with pytest.raises(ValueError, match="workspace"):
            W.wq_kv_attention(*args, workspace=bad)


def _padded(t, n):
    """t between n rows of other memory on either side, and the whole."""
    whole = torch.full((t.shape[0] + 2 * n, *t.shape[1:]), 7, dtype=t.dtype, device=t.device)
    return whole[n:n + t.shape[0]], whole


@pytest.mark.parametrize("ql", [[1, 1, 5], [40, 2, 90]])
def test_workspace_of_the_caller(W, ql):
    """The bytes asked for are enough, whatever they hold; one less is refused; nothing beside them changes."""
    banner("kv attention: caller's workspace", ql)
    q, cu, kv, cache, table = _spread_problem(37, 8, 2, 128, 64, ql, [900, 4000, 3000])
    x = dev_bf16(bf16_round(q))
    args = (x, *[dev_u8(c) for c in cache], _i32(table), _i32(cu), _i32(kv))
    want, want_lse = W.wq_kv_attention(*args, return_lse=True)
    need = W.wq_kv_attention_workspace_size(3, len(q), 0, 8, 2, 128, 64, table.shape[1])
    assert need > 0
    for fill in (0x00, 0xFF, 0x7F, 0x01):
        whole = torch.full((need + 1024,), fill, dtype=torch.uint8, device="cuda")
        for _ in range(2):                                     # as the call before left it
            got, lse = W.wq_kv_attention(*args, return_lse=True, workspace=whole[512:512 + need])
            assert torch.equal(got, want) and torch.equal(lse, want_lse)
        assert (whole[:512] == fill).all() and (whole[512 + need:] == fill).all()
    with pytest.raises(ValueError):
        W.wq_kv_attention(*args, workspace=whole[512:512 + need - 1])


def test_lengths_outside_the_contract_stay_inside_the_outputs(W):
    """Row ranges that decrease, overlap or leave the arrays: nothing beside the outputs changes."""
    banner("kv attention: row ranges that do not fit, outputs inside larger memory")
    q, cu, kv, cache, table = _spread_problem(38, 4, 2, 64, 16, [2, 3, 1, 2], [40, 20, 9, 30], spare_cols=0)
    x = dev_bf16(bf16_round(q))
    dev = [dev_u8(c) for c in cache]
    for bad in ([0, 2, 5, 4, 100], [-3, 2, 5, 6, 8], [0, 2 ** 31 - 1, 5, 6, 8], [5, 4, 3, 2, 1]):
        for hint in (0, 1):
            out, whole = _padded(x, 64)
            W.wq_kv_attention(x, *dev, _i32(table), _i32(bad), _i32(kv), max_q=hint, out=out)
            torch.cuda.synchronize()
            assert (whole[:64] == 7).all() and (whole[64 + len(q):] == 7).all()


# ---------------------------------------------------------------------------
# weights spread over many tokens
# ---------------------------------------------------------------------------
def _effective(q, cu, kv, cache, table, window=0):
    """Median over requests of the tokens that the last row's softmax is spread over, 1 / sum p^2."""
    N, H, P, D = cache[0].shape
    n = []
    for i, m in enumerate(kv):
        if m == 0 or cu[i + 1] == cu[i]:
            continue
        pages = table[i, :-(-m // P)]
        k = OK.e4m3_decode(cache[0][pages, 0]) * OK.e8m0_decode(cache[1][pages, 0])[:, None, None]
        k = k.reshape(-1, D)[max(0, m - window) if window else 0:m]
        s = k @ q[cu[i + 1] - 1, 0] * D ** -0.5
        p = np.exp(s - s.max())
        n.append(p.sum() ** 2 / (p * p).sum())
    return float(np.median(n))


SPREAD = [
    # Hq, H, D, page, query lengths, cache lengths, spare columns, tokens that count at least
    (32, 8, 128, 64, [1] * 5, [700, 1000, 64, 65, 900], 1, 50),            # a workgroup a row tile
    (32, 8, 128, 64, [1] * 3, [700, 2000, 1500], 100, 90),                 # shares of tiles and joins
    (16, 16, 64, 16, [1] * 7, [3000, 5, 1, 900, 2048, 0, 1000], 1, 50),
    (40, 8, 128, 32, [7, 1, 2, 5], [3000, 500, 1200, 600], 1, 60),         # drafted tokens
    (24, 1, 64, 128, [1, 3], [2500, 800], 1, 90),
    (4, 2, 64, 64, [1, 1, 1, 2], [20000, 600, 900, 5000], 1, 90),          # one long context
    (8, 2, 128, 64, [200, 130], [520, 400], 1, 30),                        # prompts
    (4, 4, 64, 16, [300, 40, 1], [300, 900, 700], 1, 30),
    (8, 2, 128, 32, [40, 1, 90, 5], [3000, 700, 2500, 64], 1, 90),         # rows split over the cache
    (16, 2, 64, 128, [40, 1, 90, 5], [3000, 700, 2500, 64], 1, 90),
]


@pytest.mark.parametrize("shape", SPREAD, ids=lambda s: f"{s[0]}x{s[1]}x{s[2]}p{s[3]}")
@pytest.mark.parametrize("softcap,window", [(0.0, 0), (0.0, 640), (8.0, 0)])
def test_attention_of_spread_weights(W, shape, softcap, window):
    Hq, H, D, P, ql, kl, spare, least = shape
    banner("kv attention: spread weights", shape, softcap, window)
    q, cu, kv, cache, table = _spread_problem(36, Hq, H, D, P, ql, kl, spare_cols=spare)
    assert _effective(q, cu, kv, cache, table, window) >= (least if not window else 25)
    for hint in (0, max(ql)):
        kw = {"softcap": softcap, "window": window}
        bits, lse = _attend(W, q, cu, kv, cache, table, max_q=hint, **kw)
        _compare(bits, lse, q, cu, kv, cache, table, **kw)


@pytest.mark.parametrize("page", [16, 64])
def test_nan_value_appended_in_a_prompt(W, page):
    """Append and attention together: the tokens before a NaN value do not see it."""
    banner("kv append and attention: a NaN value in a prompt", page)
    g = torch.Generator("cuda").manual_seed(40)
    T, H, G, D, at = 90, 2, 4, 64, 50
    q = torch.randn(T, H * G, D, device="cuda", generator=g).to(torch.bfloat16)
    k, v = (torch.randn(T, H, D, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    got = []
    for x in (0.0, float("nan")):
        v[at, 1, 7] = x
        N = -(-T // page)
        c = [torch.zeros(s, dtype=torch.uint8, device="cuda") for s in ((N, H, page, D), (N, H), (N, H, D, page), (N, H))]
        table = torch.full((1, N), -1, dtype=torch.int32, device="cuda")
        slots, _, cu, kv, _ = W.wq_kv_blocks(_i32([0]), _i32([T]), _i32(np.arange(N)), table, page, T)
        W.wq_kv_append(k, v, slots, *c)
        got.append(W.wq_kv_attention(q, *c, table, cu, kv))
    want, y = got
    hit = torch.zeros_like(y, dtype=torch.bool)
    hit[at:, G:, 7] = True
    assert y[hit].isnan().all() and want.isfinite().all()
    assert torch.equal(y[~hit], want[~hit])
