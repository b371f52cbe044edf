"""GPU parity of the 4-bit cache and the rotating append where the other tests do not reach: workgroups
that take many tokens, capped scores over shares of the work, row tiles of their own by the hundred, more
row tiles than waves, and the second term of the probabilities."""
from concurrent.futures import ThreadPoolExecutor

import numpy as np
import pytest
import torch

from oracle import kv4 as O4
from oracle.formats import bf16_decode, bf16_round
from tests.gpu_helpers import banner, dev_bf16, dev_u8, host_bits16
from tests.test_gpu_kv import W, _cache, _i32, _slots  # noqa: F401 (W is a fixture)
from tests.test_gpu_kv4 import _angles, _cache4, _check_attention, _check_rotary, _problem

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# rotating append
# ---------------------------------------------------------------------------
# Tokens a workgroup: 4, doubled while there are more than 2048 workgroups (of the 8-bit cache no more
# than a page's).
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("bf16,Hq,H,D,page,rot,inter,ctx,new", [
    (True, 16, 16, 64, 128, 64, False, [7], [3500]),                  # 64 tokens
    (False, 8, 8, 128, 64, 128, True, [3, 0, 70], [2900, 17, 1400]),  # 64
    (True, 16, 16, 64, 16, 32, True, [5, 16], [860, 41]),             # 16
    (True, 4, 4, 64, 32, 64, False, [0, 31, 9], [1000, 2, 1300]),     # 16
    (True, 8, 8, 64, 16, 16, False, [13] * 3000, [1] * 3000),         # single tokens: 16, and 32 of the 4-bit cache
    (False, 8, 8, 128, 64, 96, False, [1] * 4200, [1] * 4200),        # 64 single tokens
])
def test_append_rotary_many_tokens_a_workgroup(W, bits, bf16, Hq, H, D, page, rot, inter, ctx, new):
    """Runs and single tokens over several passes of a workgroup, past its 64th lane and into the next
    one's, with tokens left out whose position has no angles: the last and the first of a page,
    so that the page still has one run, and single ones."""
    banner("kv append rotary: tokens a workgroup", bits, bf16, Hq, H, D, page, rot, inter, ctx[:3], new[:3], len(ctx))
    g = np.random.default_rng(H * D + page + len(ctx))
    slots, N = _slots(g, ctx, new, page, spare=1)
    T = len(slots)
    cs = _angles(3600, rot)
    pos = np.concatenate([c + np.arange(n) for c, n in zip(ctx, new)] + [[-1]])
    live = slots >= 0
    ends = np.nonzero(live & ((slots % page == page - 1) | (slots % page == 0) | (len(ctx) > 100)))[0]
    out = g.choice(ends, max(2, len(ends) // 7), replace=False)
    pos[out] = g.choice([-1, 3600, 1 << 30, -(1 << 31)], len(out))
    amp = np.exp2(g.integers(-3, 4, (T, H, 1)))
    k, v = ((g.standard_normal((T, H, D)) * amp).astype(np.float32) for _ in range(2))
    q = g.standard_normal((T, Hq, D)).astype(np.float32)
    cache = _cache4(g, N, H, page, D) if bits == 4 else _cache(g, N, H, page, D)
    _check_rotary(W, q, k, v, pos, cs, slots, cache, bf16, inter)


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def _kind(W, q, kv, H, page, table, most_q, window=0):
    """Whether the call joins nothing ("alone") or cuts its work into shares, as its workspace says."""
    n = W.wq_kv4_attention_workspace_size(len(kv), q.shape[0], most_q, q.shape[1], H, q.shape[2], page, table.shape[1], window)
    return "shares" if n else "alone"


@pytest.mark.parametrize("H,group,most_q,D", [(8, 2, 1, 64), (8, 2, 1, 128), (5, 3, 4, 128), (8, 4, 6, 64), (8, 4, 6, 128),
                                              (3, 16, 4, 128)])
@pytest.mark.parametrize("softcap", [3.0, 40.0])
def test_attention_capped_shares(W, H, group, most_q, D, softcap):
    """Ragged decode batches and drafted tokens with capped scores, shares that begin and end anywhere:
    16-row tiles, whose probabilities are multiplied in two terms, and tiles of 32 rows."""
    banner("kv4 attention: capped shares", H, group, most_q, D, softcap)
    g = np.random.default_rng(H + D)
    kl = np.exp(g.uniform(0, np.log(3000), 40)).astype(int)
    ql = g.integers(1, most_q + 1, 40)
    kl[[3, 17]], ql[[5, 6, 30]], kl[[9, 22]] = 0, 0, [2999, 2048]
    q, cu, kv, cache, table = _problem(24, H * group, H, D, 32, ql, kl, spare_rows=2)
    assert _kind(W, q, kv, H, 32, table, most_q) == "shares"
    for kw in ({}, {"window": 700}):
        _check_attention(W, q, cu, kv, cache, table, max_q=most_q, softcap=softcap, sm_scale=0.3, **kw)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("softcap", [0.0, 5.0])
def test_attention_capped_long_context(W, D, softcap):
    """One context beside short ones, all of whose shares are one row tile's."""
    banner("kv4 attention: capped long context", D, softcap)
    q, cu, kv, cache, table = _problem(25, 8, 2, D, 128, [1, 1, 1], [20000, 3, 900])
    assert _kind(W, q, kv, 2, 128, table, 1) == "shares"
    _check_attention(W, q, cu, kv, cache, table, poison=False, max_q=1, softcap=softcap, sm_scale=0.2)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("group,most_q", [(2, 1), (4, 6)])
@pytest.mark.parametrize("softcap,window", [(0.0, 0), (4.0, 0), (30.0, 90)])
def test_attention_row_tiles_alone_by_the_hundred(W, D, group, most_q, softcap, window):
    """More row tiles than CUs, each a workgroup's own: 40 requests, 8 heads, tables of at most 1500 tokens."""
    banner("kv4 attention: row tiles of their own", D, group, most_q, softcap, window)
    g = np.random.default_rng(D + most_q)
    kl, ql = np.exp(g.uniform(0, np.log(1500), 40)).astype(int), g.integers(1, most_q + 1, 40)
    kl[:3], ql[7] = [1499, 1, 0], 0
    q, cu, kv, cache, table = _problem(26, 8 * group, 8, D, 64, ql, kl, spare_rows=1)
    assert _kind(W, q, kv, 8, 64, table, most_q, window) == "alone"
    _check_attention(W, q, cu, kv, cache, table, max_q=most_q, softcap=softcap, window=window, sm_scale=0.3)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("softcap", [0.0, 6.0])
def test_attention_more_row_tiles_than_waves(W, D, softcap):
    """Requests beyond the waves of a head (128 at 16 heads): every wave has an entry of its own for the join."""
    banner("kv4 attention: more row tiles than waves", D, softcap)
    g = np.random.default_rng(D)
    kl = np.exp(g.uniform(0, np.log(700), 150)).astype(int)
    kl[[0, 77]] = [699, 0]
    q, cu, kv, cache, table = _problem(27, 32, 16, D, 16, [1] * 150, kl)
    assert _kind(W, q, kv, 16, 16, table, 1) == "shares"
    _check_attention(W, q, cu, kv, cache, table, max_q=1, softcap=softcap, sm_scale=0.3)


@pytest.mark.parametrize("H,group,D", [(8, 1, 64), (2, 8, 128), (8, 4, 128), (1, 16, 64)])
@pytest.mark.parametrize("softcap", [0.0, 8.0])
def test_attention_probabilities_in_two_terms(W, H, group, D, softcap):
    """Tiles of 16 rows cut into shares: the output is off by its own rounding and by what 64 bits do
    not know of, not by a rounding of the probabilities to bf16.

    The bound is the other tests' with that rounding's 2^-8 of sum w |v| taken out: what it leaves is exact
    in fp32 and is multiplied too, rounded to bf16 itself, so that 2^-8 of 2^-8 remains; the sums have twice
    as many terms.  Few tokens and small scores keep the bound's other parts below what a
    lost second term does (a table wider than the contexts gives the shares)."""
    banner("kv4 attention: probabilities in two terms", H, group, D, softcap)
    g = np.random.default_rng(28)
    kl = g.integers(5, 40, 60)
    q, cu, kv, cache, table = _problem(28, H * group, H, D, 16, [1] * 60, kl, spare_cols=300)
    assert _kind(W, q, kv, H, 16, table, 1) == "shares"
    cache[1][:], cache[3][:] = 127, g.integers(126, 129, cache[3].shape)
    bits, scale = bf16_round(q), 0.02
    ref, _, weight, spread = O4.attention(bf16_decode(bits), cu, kv, *cache, table, scale, softcap)
    got = W.wq_kv4_attention(dev_bf16(bits), *[dev_u8(c) for c in cache], _i32(table), _i32(cu), _i32(kv), sm_scale=scale,
                             softcap=softcap, max_q=1)
    torch.cuda.synchronize()
    e = (D + 16) * 2.0 ** -24 * spread + softcap * 2.0 ** -22
    rel = np.expm1(2 * e) + (2 * max(kl) + 8) * 2.0 ** -23 + 2.0 ** -20 + 2.0 ** -16
    tol = 2.0 ** -8 * np.abs(ref) + rel[..., None] * 1.01 * weight + 1e-30
    worst = (np.abs(bf16_decode(host_bits16(got)) - ref) / tol).max()
    # what the probabilities' rounding alone does to this problem passes the bound many times over
    assert worst <= 1.0, f"error / bound = {worst:.3f}"


# ---------------------------------------------------------------------------
# threads
# ---------------------------------------------------------------------------
def test_calls_from_several_threads(W):
    """Compiled calls give the interpreter's lock back, so calls of several threads are inside the library
    at once: each on a stream of its own, with outputs, workspaces and a cache of its own."""
    banner("kv4: appends and attention from four threads at once")
    g = np.random.default_rng(29)
    H, D, P, T = 2, 64, 16, 70
    slots, N = _slots(g, [5], [T], P)
    pos, cs, sl = _i32(5 + np.arange(T)), torch.from_numpy(_angles(100, D)).cuda(), torch.from_numpy(slots).cuda()
    start = [dev_u8(c) for c in _cache4(g, N, H, P, D)]
    q, cu, kv, cache, table = _problem(30, 8, 2, 128, 64, [1, 1, 5], [900, 4000, 300])
    args = (dev_bf16(bf16_round(q)), *[dev_u8(c) for c in cache], _i32(table), _i32(cu), _i32(kv))
    new = [[dev_bf16(bf16_round(g.standard_normal((T, h, D)))) for h in (4, H, H)] for _ in range(4)]

    def work(i, times):
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.default_stream())
        with torch.cuda.stream(stream):
            mine = [c.clone() for c in start]
            for _ in range(times):
                out = W.wq_kv_append_rotary(*new[i], pos, cs, sl, *mine)
                W.wq_kv4_append(new[i][2], new[i][1], sl, *mine)
                got = W.wq_kv4_attention(*args, return_lse=True)
        stream.synchronize()
        return [out, *mine, *got]

    want = [work(i, 1) for i in range(4)]
    with ThreadPoolExecutor(4) as pool:
        got = list(pool.map(lambda i: work(i, 50), range(4)))
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
