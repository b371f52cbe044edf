"""What the entry points report of errors that are not theirs, and the compiled calls over entry
points that fail or take their time."""
import json
import os
import shutil
import subprocess
import sys

import pytest
import torch

from tests.gpu_helpers import banner

pytestmark = pytest.mark.gpu

@pytest.fixture(scope="module")
def W():
    import weight_only_quantized_quant_amd as W
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return W


def _u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8, device="cuda")


def _calls(W):
    """name -> (a call that launches, the tensors that it writes).  Nothing but launches and allocations in a call."""
    g = torch.Generator("cuda").manual_seed(0)
    x = torch.randn(32, 256, device="cuda", generator=g)
    xb = x.bfloat16()
    codes, scales = W.quantize_mxfp4(x, 32)
    packed, sb = W.quantize_int4(x, 128)
    out = {}
    add = out.__setitem__
    add("quantize_e4m3", lambda: W.quantize_e4m3(x, 128))
    add("quantize_mxfp4", lambda: W.quantize_mxfp4(x, 32))
    add("quantize_nvfp4", lambda: W.quantize_nvfp4(x))
    add("quantize_mx", lambda: W.quantize_mx(x))
    add("quantize_int4", lambda: W.quantize_int4(x, 128))
    add("quantize_int4_asym", lambda: W.quantize_int4_asym(x, 128))
    add("wq_dequant", lambda: W.wq_dequant(codes, W.WQ_E2M1X2, scales, W.WQ_E8M0, 32, 32, 256))
    for m in (1, 32):
        add(f"wq_gemm of {m} rows", lambda m=m: W.wq_gemm(xb[:m], packed, W.WQ_INT4X8, sb, W.WQ_BF16, 128, 32))
    logits = torch.randn(5, 64, device="cuda", generator=g)
    add("wq_moe_route", lambda: W.wq_moe_route(logits, 8))
    heads, dim, page, tokens = 2, 64, 16, 5
    q, k, v = (torch.randn(tokens, n, dim, device="cuda", generator=g).bfloat16() for n in (4, heads, heads))
    slots, positions = torch.arange(tokens, device="cuda"), torch.arange(tokens, dtype=torch.int32, device="cuda")
    angle = torch.randn(8, dim // 2, device="cuda", generator=g)
    cos_sin = torch.cat([angle.cos(), angle.sin()], 1)
    c8 = [_u8(1, heads, page, dim), _u8(1, heads), _u8(1, heads, dim, page), _u8(1, heads)]
    c4 = [_u8(1, heads, page, dim // 2), _u8(1, heads, dim // 32, page), _u8(1, heads, dim // 2, page), _u8(1, heads, dim // 32, page)]
    table, cu, lens = (torch.tensor(t, dtype=torch.int32, device="cuda") for t in ([[0]], [0, tokens], [tokens]))
    free = torch.tensor([0], dtype=torch.int32, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    spare = torch.full((1, 1), -1, dtype=torch.int32, device="cuda")
    add("wq_kv_blocks", lambda: W.wq_kv_blocks(zero, lens, free, spare, page, tokens))
    add("wq_kv_append", lambda: W.wq_kv_append(k, v, slots, *c8) or tuple(c8))
    add("wq_kv4_append", lambda: W.wq_kv4_append(k, v, slots, *c4) or tuple(c4))
    for name, c in (("8", c8), ("4", c4)):
        add(f"wq_kv_append_rotary, {name} bits",
            lambda c=c: (W.wq_kv_append_rotary(q, k, v, positions, cos_sin, slots, *c), *c))
    add("wq_kv_attention", lambda: W.wq_kv_attention(q, *c8, table, cu, lens))
    add("wq_kv4_attention", lambda: W.wq_kv4_attention(q, *c4, table, cu, lens))
    add("wq_util_spin", lambda: W.wq_util_spin(1))
    return out


def test_an_earlier_error_is_not_reported(W):
    """An error that another HIP call of the thread left belongs to that call: the next launches raise
    nothing and give what they give without it."""
    banner("errors: left by an earlier HIP call")
    here = torch.cuda.current_device()
    bad = []
    for name, f in _calls(W).items():
        banner("errors:", name)
        want = f()
        want = [t.clone() for t in (want if isinstance(want, tuple) else (want,)) if torch.is_tensor(t)]
        torch.cuda.synchronize()
        assert W.lib.hipSetDevice(100000) != 0              # no such device
        try:
            got = f()
        except RuntimeError as e:
            bad.append(f"{name}: {e}")
            got = None
        W.lib.hipGetLastError()
        torch.cuda.set_device(here)
        torch.cuda.synchronize()
        if got is not None:
            got = [t for t in (got if isinstance(got, tuple) else (got,)) if torch.is_tensor(t)]
            assert len(got) == len(want) and all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want)), name
    assert not bad, bad


# Entry points in place of the library's, which the compiled calls find first because they are loaded
# into the process's own scope before them.  The calls through ctypes are the library's still.
STUB = r"""
#include <unistd.h>
static int calls;
int stub_calls(void) { return calls; }
int wq_kv_append_rotary(void) { calls++; return 4; }
int wq_kv4_append(void) { usleep(400000); return 0; }
int wq_kv4_attention(void) { usleep(400000); return 0; }
"""
CHILD = r"""
import ctypes, json, sys, threading, time
stub = ctypes.CDLL(sys.argv[1], ctypes.RTLD_GLOBAL)
import torch
import weight_only_quantized_quant_amd as W
heads, dim, page, tokens = 2, 64, 16, 5
q, k, v = (torch.randn(tokens, n, dim, device="cuda").bfloat16() for n in (4, heads, heads))
slots, positions = torch.arange(tokens, device="cuda"), torch.arange(1, tokens + 1, dtype=torch.int32, device="cuda")
cos_sin = torch.cat([torch.zeros(8, dim // 2, device="cuda"), torch.ones(8, dim // 2, device="cuda")], 1)
shapes = ((1, heads, page, dim // 2), (1, heads, dim // 32, page), (1, heads, dim // 2, page), (1, heads, dim // 32, page))
cache = [torch.zeros(s, dtype=torch.uint8, device="cuda") for s in shapes]
table, cu, lens = (torch.tensor(t, dtype=torch.int32, device="cuda") for t in ([[0]], [0, tokens], [tokens]))
before = q.clone()
torch.cuda.synchronize()
said = None
try:
    W.wq_kv_append_rotary(q, k, v, positions, cos_sin, slots, *cache, q_out=q)
except W.WQError as e:
    said = str(e)
torch.cuda.synchronize()
got = {"said": said, "calls": stub.stub_calls(), "queries": torch.equal(q, before), "cache": not any(c.any().item() for c in cache)}
ticks, stop = [], threading.Event()
def tick():
    while not stop.is_set():
        ticks.append(time.monotonic())
        time.sleep(0.001)
t = threading.Thread(target=tick)
t.start()
for name, call in (("append", lambda: W.wq_kv4_append(k, v, slots, *cache)),
                   ("attention", lambda: W.wq_kv4_attention(q, *cache, table, cu, lens))):
    start = time.monotonic()
    call()
    got[name + " us"] = int(1e6 * (time.monotonic() - start))
    got[name] = sum(start + 0.1 < x < start + 0.3 for x in ticks)
stop.set()
t.join()
print(json.dumps(got))
"""


@pytest.fixture(scope="module")
def child(W, tmp_path_factory):
    """What a process says whose compiled calls reach the entry points above."""
    where = tmp_path_factory.mktemp("stub")
    (where / "stub.c").write_text(STUB)
    subprocess.run([shutil.which("gcc") or "cc", "-shared", "-fPIC", "-o", str(where / "stub.so"), str(where / "stub.c")], check=True)
    (where / "child.py").write_text(CHILD)
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    banner("errors: a process with entry points that fail or sleep")
    paths = os.pathsep.join(p for p in (root, os.environ.get("PYTHONPATH")) if p)
    run = subprocess.run([sys.executable, str(where / "child.py"), str(where / "stub.so")], cwd=root, capture_output=True, text=True,
                         timeout=100, env={**os.environ, "PYTHONPATH": paths})
    assert run.returncode == 0, run.stderr[-2000:]
    return json.loads(run.stdout.splitlines()[-1])


def test_a_launch_that_fails_is_not_made_again(child):
    """The compiled call raises what the entry point said and does not go the other way, where queries in
    place would be turned by a call that has failed."""
    assert child["said"] and "wq_kv_append_rotary" in child["said"] and "WQ_EHIP" in child["said"]
    assert child["calls"] == 1 and child["queries"] and child["cache"]


@pytest.mark.parametrize("name", ["append", "attention"])
def test_other_threads_run_during_a_launch(child, name):
    """An entry point that waits for 0.4 s: another thread, which ticks every millisecond, goes on."""
    assert child[name + " us"] >= 400000, "the call did not reach the stub"
    assert child[name] >= 20
