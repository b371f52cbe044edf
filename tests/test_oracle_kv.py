"""The definitions of the 8-bit key/value cache against brute force, closed
forms and invariants (CPU only)."""
import numpy as np
import pytest

from oracle import kv as OK
from oracle.e4m3 import e4m3_from_f32
from oracle.formats import e4m3_decode, e8m0_decode


def test_cover_code_is_the_least_power_of_two_that_holds_the_maximum():
    g = np.random.default_rng(0)
    a = np.concatenate([np.exp2(g.uniform(-140, 127, 4000)), 448 * np.exp2(np.arange(-120.0, 100.0)),
                        np.nextafter(np.float32(448) * np.exp2(np.arange(-110, 100)).astype(np.float32), np.float32(np.inf)),
                        [2.0 ** -149, 3.4028234663852886e38]]).astype(np.float32).astype(np.float64)
    c = OK.cover_code(a)
    assert (a <= 448 * e8m0_decode(c)).all()
    assert ((c == 0) | (a > 448 * e8m0_decode(np.maximum(c - 1, 0)))).all()
    assert OK.cover_code(0.0) == 0
    assert OK.cover_code(448.0) == 127 and OK.cover_code(449.0) == 128


@pytest.mark.parametrize("values", [False, True])
def test_append_one_run_or_token_by_token(values):
    """Whatever the runs, the scale covers the page's maximum and every element is within half an
    E4M3 step of the page's scale per rounding it saw."""
    g = np.random.default_rng(1)
    H, P, D, T = 2, 16, 64, 24
    x = g.standard_normal((T, H, D)).astype(np.float32) * np.exp2(np.arange(T) % 7)[:, None, None]
    slots = np.concatenate([3 * P + np.arange(P), 1 * P + np.arange(T - P)])
    shape = (5, H, D, P) if values else (5, H, P, D)
    empty, scales = np.zeros(shape, np.uint8), np.zeros((5, H), np.uint8)
    whole = OK.append(x, slots, empty, scales, values)
    steps = (empty, scales)
    for t in range(T):
        steps = OK.append(x[t:t + 1], slots[t:t + 1], *steps, values)
    assert np.array_equal(whole[1], steps[1])              # the scale does not depend on the runs
    for codes, sc in (whole, steps):
        for pg, rows in ((3, range(P)), (1, range(P, T))):
            v = e4m3_decode(codes[pg]) * e8m0_decode(sc[pg])[:, None, None]
            v = v.transpose(0, 2, 1) if values else v      # [H, P, D]
            for o, t in enumerate(rows):
                unit = e8m0_decode(sc[pg])[:, None]
                # at most 7 roundings, each half a step: 2^-4 relative or 2^-10 of the scale
                tol = 7 * (2.0 ** -4 * np.abs(x[t]) + 2.0 ** -10 * unit)
                assert (np.abs(v[:, o] - x[t]) <= tol).all()
    one = OK.append(x[:P], slots[:P], empty, scales, values)
    c = OK.cover_code(np.abs(x[:P]).max(axis=(0, 2)))
    got = one[0][3].transpose(0, 2, 1) if values else one[0][3]
    assert np.array_equal(got, e4m3_from_f32(np.ldexp(x[:P], 127 - c[None, :, None]).astype(np.float32)).transpose(1, 0, 2))


def test_append_skips_and_keeps():
    x = np.ones((4, 1, 64), np.float32)
    codes = np.full((2, 1, 16, 64), 0x11, np.uint8)
    scales = np.full((2, 1), 130, np.uint8)
    c, s = OK.append(x, np.array([-1, 5, 99, 18]), codes, scales, False)
    assert (c[0, 0, :5] == 0x11).all() and (c[0, 0, 6:] == 0x11).all() and s[0, 0] == 130
    assert (e4m3_decode(c[0, 0, 5]) * 8 == 1).all() and (e4m3_decode(c[1, 0, 2]) * 8 == 1).all()
    # NaN and infinities are stored, not scaled by
    x[1, 0, :3] = [np.nan, np.inf, -np.inf]
    c, s = OK.append(x[1:2], np.array([16]), codes, scales, False)
    assert list(c[1, 0, 0, :3]) == [0x7F, 0x7E, 0xFE] and s[1, 0] == OK.cover_code(1.0)


def test_blocks_by_hand():
    table = np.full((3, 4), -1)
    table[1, :2] = [7, 8]
    t, slots, pos, cu, kv, state = OK.blocks([0, 20, 0], [17, 13, 40], [5, 6, 9, 2, 3], 0, 16, table, 32)
    assert t[0].tolist() == [5, 6, -1, -1] and t[1].tolist() == [7, 8, 9, -1]
    assert slots[:17].tolist() == [5 * 16 + i for i in range(16)] + [6 * 16]
    assert slots[17:30].tolist() == [8 * 16 + 4 + i for i in range(12)] + [9 * 16]
    assert slots[30:].tolist() == [-1, -1] and pos[17] == 20
    # 40 more tokens pass row 32: refused, though two pages are left for its three
    assert cu.tolist() == [0, 17, 30, 32] and kv.tolist() == [17, 33, 0] and state.tolist() == [3, 1]


def test_attention_closed_forms():
    H, P, D = 1, 16, 64
    one = e4m3_from_f32(np.ones(1, np.float32))[0]
    k = np.zeros((3, H, P, D), np.uint8)                   # all scores 0: the mean of what is seen
    v = np.zeros((3, H, D, P), np.uint8)
    ks = vs = np.full((3, H), 127, np.uint8)
    for pg in range(3):
        v[pg] = e4m3_from_f32(np.arange(P, dtype=np.float32) + 16 * pg)[None, None]
    vs = np.full((3, H), 128, np.uint8)
    q = np.ones((3, 2, D))
    table = np.array([[2, 0, -1], [1, -1, -1]])
    out, lse, _, _ = OK.attention(q, [0, 2, 3], [18, 0], k, ks, v, vs, table, 1.0)
    val = 2 * e4m3_decode(np.concatenate([v[2, 0, 0], v[0, 0, 0]]))
    assert np.allclose(out[0], val[:17].mean()) and np.allclose(out[1], val[:18].mean())
    assert np.allclose(lse[:2], np.log([[17, 17], [18, 18]]))
    assert (out[2] == 0).all() and np.isneginf(lse[2]).all()   # nothing to see
    out, lse, _, _ = OK.attention(q, [0, 2, 3], [18, 1], k, ks, v, vs, table, 1.0, window=3)
    assert np.allclose(out[1], val[15:18].mean()) and np.allclose(lse[1], np.log(3))
    k[2, 0, 4] = one                                        # one key with score 64 * sm, capped
    out, lse, _, _ = OK.attention(q[:1], [0, 1], [16], k, ks, v, vs, table[:1], 0.5, softcap=4.0)
    assert np.allclose(lse, np.log(15 + np.exp(4 * np.tanh(32 / 4))))
