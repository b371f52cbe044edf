"""The definitions of the 4-bit key/value cache and of the rotation against
closed forms, brute force and the 8-bit definitions (CPU only)."""
import numpy as np
import pytest

from oracle import kv as OK
from oracle import kv4 as O4
from oracle.e4m3 import e4m3_from_f32
from oracle.formats import E2M1_GRID, e8m0_decode
from oracle.mxfp4 import quantize_mxfp4


def test_quantize_is_mxfp4():
    g = np.random.default_rng(0)
    x = (g.standard_normal((40, 3, 128)) * np.exp2(g.integers(-30, 30, (40, 3, 1)))).astype(np.float32)
    codes, scales = O4.quantize(x)
    want, c = quantize_mxfp4(x.reshape(-1, 128), 32)
    assert np.array_equal(codes.reshape(-1, 64), want) and np.array_equal(scales.reshape(-1, 4), c)


def test_quantize_special_values():
    x = np.zeros((5, 32), np.float32)
    x[0, :4] = [np.nan, -np.nan, np.inf, -np.inf]           # alone: scale of zeros
    x[1, :3] = [np.nan, np.inf, 1.0]                        # beside a finite one, which sets the scale
    x[2, :2] = [3.4e38, -3.4e38]
    x[3, :2] = [-0.0, 1e-45]
    codes, scales = O4.quantize(x)
    assert codes[0, :2].tolist() == [0, 7 | 15 << 4] and scales[0, 0] == 0
    assert codes[1, :2].tolist() == [7 << 4, 6] and scales[1, 0] == 125    # 1 = 4 * 2^-2
    assert scales[2, 0] == 252 and codes[2, 0] == 7 | 15 << 4              # 3.4e38 = 8 * 2^125, saturated
    assert codes[3, 0] == 8 and scales[3, 0] == 0
    assert (codes[4] == 0).all() and scales[4, 0] == 0


def test_append_and_dequant():
    """Every token comes back within half an E2M1 step of its block, wherever its slot is, and no
    other byte changes."""
    g = np.random.default_rng(1)
    N, H, P, D, T = 4, 2, 16, 64, 30
    x = g.standard_normal((T, H, D)).astype(np.float32)
    slots = g.permutation(N * P)[:T]
    slots[[3, 9]] = [-1, N * P]
    for values in (False, True):
        codes = np.full((N, H, D // 2, P) if values else (N, H, P, D // 2), 0xA5, np.uint8)
        scales = np.full((N, H, D // 32, P), 77, np.uint8)
        c, s = O4.append(x, slots, codes, scales, values)
        got = O4.dequant(c, s, values)
        used = np.zeros(N * P, bool)
        for t, sl in enumerate(slots):
            if not 0 <= sl < N * P:
                continue
            used[sl] = True
            v, unit = got[sl // P, :, sl % P], np.repeat(e8m0_decode(s[sl // P, :, :, sl % P]), 32, axis=1)
            # values of up to 4 are half a step of 1 off at most, those of up to 6 (and the saturated
            # ones of up to 7) a whole 1
            assert (np.abs(v - x[t]) <= np.where(np.abs(x[t]) <= 4 * unit, 0.5, 1.0) * unit).all()
        free = ~used.reshape(N, P)
        assert (s.transpose(0, 3, 1, 2)[free] == 77).all()
        rows = c.transpose(0, 3, 1, 2) if values else c.transpose(0, 2, 1, 3)
        assert (rows[free] == 0xA5).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotate_is_a_rotation(interleaved):
    """Lengths of pairs stay, angles add, channels behind `rot` and tokens without an angle stay."""
    g = np.random.default_rng(2)
    T, D, rot = 6, 64, 32
    x = g.standard_normal((T, 2, D))
    ang = np.arange(50)[:, None] * 0.1 ** (np.arange(rot // 2) / 8)
    cs = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    y = O4.rotate(x, [3, 7, 0, 49, 50, -1], cs, interleaved)
    assert np.array_equal(y[..., rot:], x[..., rot:]) and np.array_equal(y[[2, 4, 5]], x[[2, 4, 5]])
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    z, w = x[..., a] + 1j * x[..., b], y[..., a] + 1j * y[..., b]
    assert np.allclose(w[:2], z[:2] * np.exp(1j * ang[[3, 7]])[:, None])
    assert np.allclose(O4.rotate(O4.rotate(x, [3] * T, cs, interleaved), [4] * T, cs, interleaved),
                       O4.rotate(x, [7] * T, cs, interleaved))


def test_attention_agrees_with_the_8_bit_definition():
    """A cache that both formats hold exactly: the same results."""
    g = np.random.default_rng(3)
    N, H, P, D = 5, 2, 16, 64
    n = g.integers(0, 16, (2, N, H, P, D))
    val = E2M1_GRID[n & 7] * np.where(n & 8, -1.0, 1.0)
    packed = (n[..., 0::2] | n[..., 1::2] << 4).astype(np.uint8)
    s4 = np.full((N, H, D // 32, P), 126, np.uint8)
    c8 = e4m3_from_f32(val.astype(np.float32))
    s8 = np.full((N, H), 126, np.uint8)
    q = g.standard_normal((7, 4, D))
    table = np.array([[3, 1, 0], [2, -1, 4]])
    args = ([0, 4, 7], [40, 46])
    for kw in ({}, {"softcap": 2.0}, {"window": 11}):
        a = O4.attention(q, *args, packed[0], s4, packed[1].transpose(0, 1, 3, 2), s4, table, 0.2, **kw)
        b = OK.attention(q, *args, c8[0], s8, c8[1].transpose(0, 1, 3, 2), s8, table, 0.2, **kw)
        for x, y in zip(a, b):
            assert np.allclose(x, y, rtol=1e-12, atol=1e-13)
