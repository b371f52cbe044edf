"""GPU parity of the rotating append where the other tests do not reach: workgroups that take many tokens."""
import numpy as np
import pytest

from tests.gpu_helpers import banner
from tests.test_gpu_kv import W, _cache, _slots  # noqa: F401 (W is a fixture)
from tests.test_gpu_kv4 import _angles, _cache4, _check_rotary

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
