"""Refusals of the 4-bit cache's entry points and of the rotating append: on the
host, before any launch (CPU only)."""
import os
import shutil
import subprocess
import sys

import pytest
import torch

P, P2, ODD = 0x10000, 0x20000, 0x10004                     # never dereferenced


@pytest.fixture(scope="module")
def lib():
    import weight_only_quantized_quant_amd as W            # sets the argument types
    return W.lib


def test_append_refusals(lib):
    def call(k=P, ks=512, v=P, vs=512, dt=1, slots=P, tokens=4, heads=4, dim=128, page=64, pages=10, kc=P, ksc=P, vc=P,
             vsc=P):
        return lib.wq_kv4_append(k, ks, v, vs, dt, slots, tokens, heads, dim, page, pages, kc, ksc, vc, vsc, None)
    assert call(dt=2) == 3 and call(dim=96) == 3 and call(dim=256) == 3 and call(page=24) == 3
    for bad in ({"tokens": -1}, {"heads": 0}, {"heads": 1 << 20}, {"pages": 0}, {"k": None}, {"v": None},
                {"slots": None}, {"kc": None}, {"ksc": None}, {"vc": None}, {"vsc": None}, {"ks": 504}, {"vs": 256},
                {"ks": 516}, {"vs": 1 << 41}, {"pages": 1 << 40}, {"tokens": 1 << 31}):
        assert call(**bad) == 1, bad
    for bad in ("k", "v", "kc", "vc", "ksc", "vsc"):
        assert call(**{bad: ODD}) == 2, bad
    assert call(tokens=0, k=None, v=None, slots=None) == 0   # nothing to write


@pytest.mark.parametrize("cache", [2, 3])
def test_rotary_refusals(lib, cache):
    def call(q=P, qs=1024, hq=8, k=P, ks=512, v=P, vs=512, dt=1, pos=P, cs=P, max_pos=100, rot=128, inter=0, slots=P,
             tokens=4, heads=4, dim=128, cd=cache, page=64, pages=10, kc=P, ksc=P, vc=P, vsc=P, out=P2, os=1024):
        return lib.wq_kv_append_rotary(q, qs, hq, k, ks, v, vs, dt, pos, cs, max_pos, rot, inter, slots, tokens, heads,
                                       dim, cd, page, pages, kc, ksc, vc, vsc, out, os, None)
    for bad in ({"dt": 2}, {"dim": 96}, {"page": 24}, {"cd": 0}, {"cd": 4}, {"rot": 0}, {"rot": 8}, {"rot": 24},
                {"rot": 144}, {"rot": 128, "dim": 64, "ks": 256, "vs": 256, "qs": 512, "os": 512}, {"rot": -16}):
        assert call(**bad) == 3, bad
    for bad in ({"tokens": -1}, {"heads": 0}, {"pages": 0}, {"k": None}, {"v": None}, {"slots": None}, {"kc": None},
                {"ksc": None}, {"vc": None}, {"vsc": None}, {"ks": 504}, {"vs": 516}, {"pos": None}, {"cs": None},
                {"max_pos": 0}, {"max_pos": 1 << 40}, {"hq": -1}, {"hq": 1 << 20}, {"q": None}, {"out": None},
                {"qs": 1016}, {"os": 1016}, {"qs": 1028}, {"os": 1028}, {"qs": 1 << 41}, {"os": 1 << 41},
                {"out": P, "os": 2048}, {"out": P, "dt": 0}):
        assert call(**bad) == 1, bad
    for bad in ("q", "k", "v", "kc", "vc", "cs"):
        assert call(**{bad: ODD}) == 2, bad
    assert call(out=P2 + 4) == 2
    assert call(tokens=0) == 0 and call(tokens=0, q=None, out=None, hq=0, qs=0, os=0) == 0


@pytest.mark.parametrize("cache", [2, 3])
def test_rotary_refuses_an_output_that_is_another_argument(lib, cache):
    """Keys, values, indices, angles and the cache are read or written while the queries are written."""
    where = {n: 0x100000 * (i + 1) for i, n in enumerate(("q", "k", "v", "pos", "cs", "slots", "kc", "ksc", "vc", "vsc"))}

    def call(out):
        w = where
        return lib.wq_kv_append_rotary(w["q"], 1024, 8, w["k"], 1024, w["v"], 1024, 1, w["pos"], w["cs"], 100, 128, 0,
                                       w["slots"], 4, 8, 128, cache, 64, 10, w["kc"], w["ksc"], w["vc"], w["vsc"], out, 1024, None)
    for name in where:
        if name != "q":
            assert call(where[name]) == 1, name


def test_attention_refusals(lib):
    def call(q=P, qs=1024, cu=P, kv=P, batch=2, tokens=4, max_q=0, hq=8, hk=4, dim=128, kc=P, ksc=P, vc=P, vsc=P,
             page=64, pages=10, table=P, width=4, sm=0.1, cap=0.0, window=0, out=P2, lse=None, ws=P, wsb=1 << 40):
        return lib.wq_kv4_attention(q, qs, cu, kv, batch, tokens, max_q, hq, hk, dim, kc, ksc, vc, vsc, page, pages,
                                    table, width, sm, cap, window, out, lse, ws, wsb, None)
    assert call(dim=32) == 3 and call(page=20) == 3
    assert call(cap=2000.0) == 3 and call(cap=1e-4) == 3 and call(cap=1.0, sm=20000.0) == 3 and call(sm=1.8e38) == 3
    inf, nan = float("inf"), float("nan")
    for bad in ({"batch": -1}, {"tokens": -1}, {"max_q": -1}, {"hk": 0}, {"hq": 6}, {"hq": 2}, {"pages": 0},
                {"width": 0}, {"width": 1 << 26}, {"window": -1}, {"sm": 0.0}, {"sm": -1.0}, {"sm": inf}, {"sm": nan},
                {"cap": -1.0}, {"cap": inf}, {"cap": nan}, {"qs": 1000}, {"qs": 1028}, {"q": None}, {"cu": None},
                {"kv": None}, {"table": None}, {"out": None}, {"kc": None}, {"ksc": None}, {"vc": None},
                {"vsc": None}, {"tokens": 1 << 31}, {"tokens": (1 << 31) - 200}, {"pages": 1 << 40}, {"out": P}):
        assert call(**bad) == 1, bad
    for bad in ("q", "out", "kc", "vc", "ksc", "vsc", "ws"):
        assert call(**{bad: ODD}) == 2, bad
    assert call(batch=0) == 0 and call(tokens=0) == 0        # nothing to compute


def test_attention_workspace_is_asked_for(lib):
    size = lib.wq_kv4_attention_workspace_size
    ok = (3, 3, 1, 32, 8, 128, 64, 512, 0)
    need = size(*ok)
    call = lambda wsb, ws=P: lib.wq_kv4_attention(P, 4096, P, P, 3, 3, 1, 32, 8, 128, P, P, P, P, 64, 10, P, 512, 0.1,
                                                  0.0, 0, P2, None, ws, wsb, None)
    if need > 0:
        assert call(need - 1) == 1 and call(need, None) == 1
    for bad in ((-1, 3, 1, 32, 8, 128, 64, 512, 0), (3, -3, 1, 32, 8, 128, 64, 512, 0), (3, 3, 1, 30, 8, 128, 64, 512, 0),
                (3, 3, 1, 32, 0, 128, 64, 512, 0), (3, 3, 1, 32, 8, 100, 64, 512, 0), (3, 3, 1, 32, 8, 128, 7, 512, 0),
                (3, 3, 1, 32, 8, 128, 64, 0, 0), (3, 3, 1, 32, 8, 128, 64, 512, -1)):
        assert size(*bad) == 0, bad


def test_binding_refuses_host_tensors():
    import weight_only_quantized_quant_amd as W
    i = torch.zeros(2, dtype=torch.int32)
    x = torch.zeros(2, 1, 64, dtype=torch.bfloat16)
    c, s = torch.zeros(2, 1, 16, 32, dtype=torch.uint8), torch.zeros(2, 1, 2, 16, dtype=torch.uint8)
    v = c.transpose(2, 3).contiguous()
    with pytest.raises(ValueError, match="k must"):
        W.wq_kv4_append(x, x, i.long(), c, s, v, s)
    with pytest.raises(ValueError, match="k must"):
        W.wq_kv_append_rotary(x, x, x, i, torch.zeros(9, 64), i.long(), c, s, v, s)
    with pytest.raises(ValueError, match="q must"):
        W.wq_kv4_attention(x, c, s, v, s, i.view(2, 1), torch.zeros(3, dtype=torch.int32), i)


def test_a_package_without_its_compiled_calls_says_so(tmp_path):
    import weight_only_quantized_quant_amd as W
    here, name = os.path.dirname(W.__file__), "weight_only_quantized_quant_amd"
    (tmp_path / name).mkdir()
    shutil.copy(os.path.join(here, "__init__.py"), tmp_path / name)
    os.symlink(os.path.join(here, "libwq.so"), tmp_path / name / "libwq.so")
    got = subprocess.run([sys.executable, "-c", f"import {name}"], cwd=tmp_path, capture_output=True, text=True,
                         env={**os.environ, "PYTHONPATH": str(tmp_path)})
    assert got.returncode != 0 and "_calls.so is missing: build it with" in got.stderr


@pytest.mark.parametrize("why", ["not loadable", "other torch"])
def test_compiled_calls_that_do_not_fit_the_process(tmp_path, why):
    """The package works as it does without them, by ctypes, and says so once."""
    import weight_only_quantized_quant_amd as W
    here, name = os.path.dirname(W.__file__), "weight_only_quantized_quant_amd"
    (tmp_path / name).mkdir()
    shutil.copy(os.path.join(here, "__init__.py"), tmp_path / name)
    os.symlink(os.path.join(here, "libwq.so"), tmp_path / name / "libwq.so")
    if why == "other torch":
        os.symlink(os.path.join(here, "_calls.so"), tmp_path / name / "_calls.so")
    else:
        (tmp_path / name / "_calls.so").write_bytes(b"no library")
    (tmp_path / "child.py").write_text(f"""
import warnings
import torch
if {why == "other torch"}:
    torch.__version__ = "1.0"
with warnings.catch_warnings(record=True) as got:
    warnings.simplefilter("always")
    import {name} as W
assert [w.category for w in got] == [RuntimeWarning] and "ctypes" in str(got[0].message), got
assert W._calls.kv4_append(1, 2) is W._calls.kv_append_rotary() is W._calls.kv4_attention(3) is NotImplemented
assert W.lib.wq_kv4_attention_workspace_size(3, 3, 1, 32, 8, 128, 64, 512, 0) > 0
x, i = torch.zeros(2, 1, 64, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int64)
c, s = torch.zeros(2, 1, 16, 32, dtype=torch.uint8), torch.zeros(2, 1, 2, 16, dtype=torch.uint8)
try:
    W.wq_kv4_append(x, x, i, c, s, c.transpose(2, 3).contiguous(), s)
except ValueError as e:
    assert "k must" in str(e)
else:
    raise AssertionError("host tensors were taken")
print(got[0].message)
""")
    got = subprocess.run([sys.executable, str(tmp_path / "child.py")], cwd=tmp_path, capture_output=True, text=True,
                         env={**os.environ, "PYTHONPATH": str(tmp_path)})
    assert got.returncode == 0, got.stderr
    assert (why != "other torch") or "built for torch" in got.stdout


def test_compiled_calls_that_fit_load_without_a_warning():
    import weight_only_quantized_quant_amd as W
    got = subprocess.run([sys.executable, "-W", "error::RuntimeWarning", "-c", "import weight_only_quantized_quant_amd as W; print(W._calls.__file__)"],
                         cwd=os.path.dirname(os.path.dirname(W.__file__)), capture_output=True, text=True)
    assert got.returncode == 0 and "_calls.so" in got.stdout, got.stderr
