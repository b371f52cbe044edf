"""Refusals of the key/value cache entry points: on the host, before any
launch (CPU only)."""
import ctypes
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "weight_only_quantized_quant_amd", "libwq.so")

P, P2, P3, ODD = 0x10000, 0x20000, 0x30000, 0x10004        # never dereferenced


@pytest.fixture(scope="module")
def lib():
    import weight_only_quantized_quant_amd as W            # sets the argument types
    return W.lib


def test_blocks_refusals(lib):
    def call(page=64, batch=4, width=8, tokens=4, num_free=3, ctx=P, new=P, free=P, cur=None, table=P2, slots=P3,
             pos=P3 + 64, cu=P3 + 128, kv=P3 + 192, state=P3 + 256):
        return lib.wq_kv_blocks(ctx, new, batch, free, num_free, cur, page, table, width, tokens, slots, pos, cu, kv,
                                state, None)
    assert call(page=48) == 3 and call(page=8) == 3 and call(page=256) == 3 and call(page=0) == 3
    for bad in ({"batch": -1}, {"width": 0}, {"tokens": -1}, {"num_free": -1}, {"ctx": None}, {"new": None},
                {"free": None}, {"table": None}, {"slots": None}, {"pos": None}, {"cu": None}, {"kv": None},
                {"state": None}, {"batch": 1 << 31}, {"width": 1 << 31}, {"tokens": 1 << 31}, {"num_free": 1 << 31},
                {"batch": 1 << 30, "width": 1 << 30}):
        assert call(**bad) == 1, bad
    for alias in ({"kv": P}, {"cu": P}, {"state": P}, {"cur": P3 + 256}, {"cur": P3 + 128}, {"table": P}):
        assert call(**alias) == 1, alias


def test_append_refusals(lib):
    def call(k=P, ks=512, v=P, vs=512, dt=1, slots=P, tokens=4, heads=4, dim=128, page=64, pages=10, kc=P, ksc=P, vc=P,
             vsc=P):
        return lib.wq_kv_append(k, ks, v, vs, dt, slots, tokens, heads, dim, page, pages, kc, ksc, vc, vsc, None)
    assert call(dt=2) == 3 and call(dim=96) == 3 and call(dim=256) == 3 and call(page=24) == 3
    for bad in ({"tokens": -1}, {"heads": 0}, {"heads": 1 << 20}, {"pages": 0}, {"k": None}, {"v": None},
                {"slots": None}, {"kc": None}, {"ksc": None}, {"vc": None}, {"vsc": None}, {"ks": 504}, {"vs": 256},
                {"ks": 516}, {"vs": 1 << 41}, {"pages": 1 << 40}, {"tokens": 1 << 31}):
        assert call(**bad) == 1, bad
    for bad in ("k", "v", "kc", "vc"):
        assert call(**{bad: ODD}) == 2, bad
    assert call(tokens=0, k=None, v=None, slots=None) == 0   # nothing to write


def test_attention_refusals(lib):
    def call(q=P, qs=1024, cu=P, kv=P, batch=2, tokens=4, max_q=0, hq=8, hk=4, dim=128, kc=P, ksc=P, vc=P, vsc=P,
             page=64, pages=10, table=P, width=4, sm=0.1, cap=0.0, window=0, out=P2, lse=None, ws=P, wsb=1 << 40):
        return lib.wq_kv_attention(q, qs, cu, kv, batch, tokens, max_q, hq, hk, dim, kc, ksc, vc, vsc, page, pages,
                                   table, width, sm, cap, window, out, lse, ws, wsb, None)
    assert call(dim=32) == 3 and call(page=20) == 3
    assert call(cap=2000.0, out=P2) == 3 and call(cap=1e-4, out=P2) == 3 and call(cap=1.0, sm=20000.0) == 3
    inf, nan = float("inf"), float("nan")
    for bad in ({"batch": -1}, {"tokens": -1}, {"max_q": -1}, {"hk": 0}, {"hq": 6}, {"hq": 2}, {"pages": 0},
                {"width": 0}, {"width": 1 << 26}, {"window": -1}, {"sm": 0.0}, {"sm": -1.0}, {"sm": inf}, {"sm": nan},
                {"cap": -1.0}, {"cap": inf}, {"cap": nan}, {"qs": 1000}, {"qs": 1028}, {"q": None}, {"cu": None},
                {"kv": None}, {"table": None}, {"out": None}, {"kc": None}, {"ksc": None}, {"vc": None},
                {"vsc": None}, {"tokens": 1 << 31}, {"tokens": (1 << 31) - 200}, {"pages": 1 << 40}, {"out": P}):
        assert call(**bad) == 1, bad
    for bad in ("q", "out", "kc", "vc", "ws"):
        assert call(**{bad: ODD}) == 2, bad
    assert call(batch=0) == 0 and call(tokens=0) == 0        # nothing to compute


def test_attention_workspace_is_asked_for(lib):
    size = lib.wq_kv_attention_workspace_size
    ok = (3, 3, 1, 32, 8, 128, 64, 512, 0)
    need = size(*ok)
    args = lambda wsb, ws=P: lib.wq_kv_attention(P, 4096, P, P, 3, 3, 1, 32, 8, 128, P, P, P, P, 64, 10, P, 512, 0.1,
                                                 0.0, 0, P2, None, ws, wsb, None)
    assert need > 0 and args(need - 1) == 1 and args(need, None) == 1
    assert size(*ok[:7], 8, 0) == 0 and size(*ok[:8], 300) == 0        # short contexts and windows are not split
    # sizes the call refuses need nothing
    for bad in ((-1, 3, 1, 32, 8, 128, 64, 512, 0), (3, -3, 1, 32, 8, 128, 64, 512, 0), (3, 3, 1, 30, 8, 128, 64, 512, 0),
                (3, 3, 1, 32, 0, 128, 64, 512, 0), (3, 3, 1, 32, 8, 100, 64, 512, 0), (3, 3, 1, 32, 8, 128, 7, 512, 0),
                (3, 3, 1, 32, 8, 128, 64, 0, 0), (3, 3, 1, 32, 8, 128, 64, 512, -1)):
        assert size(*bad) == 0, bad


def test_binding_refuses_host_tensors():
    import weight_only_quantized_quant_amd as W
    i = torch.zeros(2, dtype=torch.int32)
    x = torch.zeros(2, 1, 64, dtype=torch.bfloat16)
    c, s = torch.zeros(2, 1, 16, 64, dtype=torch.uint8), torch.zeros(2, 1, dtype=torch.uint8)
    with pytest.raises(ValueError, match="ctx_lens"):
        W.wq_kv_blocks(i, i, i, i.view(2, 1), 16, 2)
    with pytest.raises(ValueError, match="k must"):
        W.wq_kv_append(x, x, i.long(), c, s, c.transpose(2, 3), s)
    with pytest.raises(ValueError, match="q must"):
        W.wq_kv_attention(x, c, s, c.transpose(2, 3), s, i.view(2, 1), torch.zeros(3, dtype=torch.int32), i)
