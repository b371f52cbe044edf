"""Measured cases of the 4-bit paged key/value cache and of the append that
rotates by position: what is written to the caches of both widths on a step,
and the attention that reads the 4-bit one.

4-bit cache: E2M1 elements, one E8M0 scale for 32 channels of one token.  A page
holds `page` tokens: keys [pages, kv_heads, page, dim / 2] bytes, values
[pages, kv_heads, dim / 2, page] bytes (transposed, the order in which the
second product reads them), channel 2j in the low nibble of byte j, and scales
[pages, kv_heads, dim / 32, page] for either.

8-bit cache: E4M3 keys [pages, kv_heads, page, dim] and values [pages, kv_heads,
dim, page], one E8M0 scale for each page and head.

Codes of the 4-bit cache are returned as they lie there, two to a byte: they are
whole numbers that have to be equal.  So that the rotated keys have one right
code each, they are taken from 64 bits, rounded once to fp32, on either side.

`run` computes each operator in elementary torch operations where `own` is
false and calls the package where it is true; `exact` is the definition in 64
bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # One decode step into the 8-bit cache: 64 requests, one token each,
        # queries and keys rotated whole.
        {"name": "rotate_step", "op": "rotate", "bits": 8, "batch": 64, "tokens": 64, "ones": True, "ctx_hi": 500,
         "far": 0, "q_heads": 32, "heads": 8, "dim": 128, "page": 64, "rot": 128, "inter": False, "f32": False},
        # Whole prompts written to the 4-bit cache.
        {"name": "rotate_prompts", "op": "rotate", "bits": 4, "batch": 6, "tokens": 8192, "ones": False, "ctx_hi": 0,
         "far": 0, "q_heads": 32, "heads": 8, "dim": 128, "page": 64, "rot": 128, "inter": False, "f32": False},
        # Chunks far inside long documents: an odd number of tokens, half of the
        # channels rotated in neighbouring pairs, inputs in 32 bits, small pages.
        {"name": "rotate_odd", "op": "rotate", "bits": 8, "batch": 11, "tokens": 1037, "ones": False, "ctx_hi": 300,
         "far": 120000, "q_heads": 6, "heads": 3, "dim": 64, "page": 16, "rot": 32, "inter": True, "f32": True},
        # One decode step of a full server into the 4-bit cache, keys as they come.
        {"name": "append4_step", "op": "append4", "batch": 128, "tokens": 128, "ones": True, "ctx_hi": 500,
         "heads": 8, "dim": 128, "page": 64, "f32": False},
        # Chunks of prompts that begin and end inside pages, heads of 64.
        {"name": "append4_chunks", "op": "append4", "batch": 9, "tokens": 8111, "ones": False, "ctx_hi": 300,
         "heads": 4, "dim": 64, "page": 32, "f32": False},
        # One request decoding alone: latency.
        {"name": "attend4_single", "op": "attend4", "batch": 1, "ones": 1, "q_lo": 1, "q_hi": 1, "kv_lo": 1000,
         "kv_hi": 1000, "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "cap": 0.0, "window": 0, "lens": 1},
        # A decode batch at ordinary contexts.
        {"name": "attend4_batch", "op": "attend4", "batch": 64, "ones": 64, "q_lo": 1, "q_hi": 1, "kv_lo": 2048,
         "kv_hi": 8192, "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "cap": 0.0, "window": 0, "lens": 2},
        # One very long context beside short ones, large pages.
        {"name": "attend4_long", "op": "attend4", "batch": 5, "ones": 5, "q_lo": 1, "q_hi": 1, "kv_lo": 200,
         "kv_hi": 131072, "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 128, "cap": 0.0, "window": 0, "lens": 3},
        # As many key heads as query heads, heads of 64, capped scores, a
        # sliding window, pages of 16, an odd batch.
        {"name": "attend4_window", "op": "attend4", "batch": 33, "ones": 33, "q_lo": 1, "q_hi": 1, "kv_lo": 1,
         "kv_hi": 5000, "q_heads": 16, "kv_heads": 16, "dim": 64, "page": 16, "cap": 30.0, "window": 1000, "lens": 4},
        # A few drafted tokens per request checked at once, five query heads
        # to a key head.
        {"name": "attend4_verify", "op": "attend4", "batch": 24, "ones": 3, "q_lo": 2, "q_hi": 7, "kv_lo": 500,
         "kv_hi": 6000, "q_heads": 40, "kv_heads": 8, "dim": 128, "page": 32, "cap": 0.0, "window": 0, "lens": 5},
        # Whole prompts against the cache they were just written to.
        {"name": "attend4_prompts", "op": "attend4", "batch": 3, "ones": 0, "q_lo": 1500, "q_hi": 4096, "kv_lo": 1500,
         "kv_hi": 4096, "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "cap": 0.0, "window": 0, "lens": 6},
        # A mixed step: chunks of long prompts beside decoding requests, with
        # capped scores.
        {"name": "attend4_chunks", "op": "attend4", "batch": 6, "ones": 4, "q_lo": 700, "q_hi": 1024, "kv_lo": 4000,
         "kv_hi": 16000, "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "cap": 50.0, "window": 0, "lens": 7},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["rotate", "rotate", "append4", "attend4", "attend4", "attend4"])
    page = rng.choice([16, 32, 64, 128])
    if kind != "attend4":
        ones = rng.random() < 0.4
        batch = _log_int(rng, 1, 128) if ones else _log_int(rng, 1, 12)
        c = {"op": kind, "batch": batch, "tokens": batch if ones else _log_int(rng, batch * 8, 8192), "ones": ones,
             "ctx_hi": rng.choice([0, 100, 500]), "heads": rng.choice([1, 2, 3, 8]), "dim": rng.choice([64, 128]),
             "page": page, "f32": rng.random() < 0.25}
        if kind == "rotate":
            c.update(bits=rng.choice([4, 8]), far=rng.choice([0, 0, 5000, 120000]),
                     q_heads=c["heads"] * rng.choice([1, 2, 4]), rot=rng.choice([16, 32, 64, c["dim"], c["dim"]]),
                     inter=rng.random() < 0.4)
        return c
    top = {"bytes": 0, "flops": 0}
    for c in listed():
        if c["op"] == "attend4":
            w = work(c)
            top = {k: max(top[k], w[k]) for k in top}
    while True:
        shape = rng.choice(["step", "step", "verify", "prompts", "chunks"])
        kv_heads = rng.choice([1, 2, 4, 8, 16])
        group = rng.choice([1, 2, 4, 5, 8])
        kv_hi = _log_int(rng, 64, 65536 if shape == "step" else 16000 if shape == "verify" else 4096)
        kv_lo = _log_int(rng, 1, kv_hi)
        batch = _log_int(rng, 1, 64 if shape == "step" else 24 if shape == "verify" else 6)
        q_hi = {"step": 1, "verify": rng.randint(2, 8), "prompts": kv_hi, "chunks": max(1, kv_hi // 2)}[shape]
        q_lo = {"step": 1, "verify": 1, "prompts": kv_lo, "chunks": max(1, q_hi // 2)}[shape]
        c = {"op": "attend4", "batch": batch, "ones": batch if shape == "step" else rng.randint(0, batch // 2),
             "q_lo": q_lo, "q_hi": q_hi, "kv_lo": kv_lo, "kv_hi": kv_hi, "q_heads": kv_heads * group,
             "kv_heads": kv_heads, "dim": rng.choice([64, 128]), "page": page, "cap": rng.choice([0.0, 0.0, 30.0, 50.0]),
             "window": rng.choice([0, 0, 0, rng.randint(1, kv_hi)]), "lens": rng.randint(0, 10 ** 6)}
        w = work(c)
        scores = batch * c["q_heads"] * q_hi * kv_hi
        if w["bytes"] <= top["bytes"] and w["flops"] <= top["flops"] and scores <= 3.2e9:
            return c


# ---------------------------------------------------------------------------
# lengths
# ---------------------------------------------------------------------------
def _attend_lens(c):
    """Query and cache lengths of an attention case (part of the case, not of the data)."""
    r = np.random.RandomState(c["lens"])
    b = c["batch"]
    kv = np.exp(r.uniform(math.log(c["kv_lo"]), math.log(c["kv_hi"]), b)).round().astype(np.int64)
    q = np.exp(r.uniform(math.log(c["q_lo"]), math.log(c["q_hi"]), b)).round().astype(np.int64)
    kv[0] = c["kv_hi"]
    q[0] = c["q_hi"]
    q[b - c["ones"]:] = 1
    return q, np.maximum(kv, q)


def _new_lens(c, r):
    """Lengths before the step and new tokens of each request for the appends."""
    b = c["batch"]
    ctx = np.exp(r.uniform(0, math.log(c["ctx_hi"]), b)).astype(np.int64) if c["ctx_hi"] else np.zeros(b, np.int64)
    if c["ones"]:
        return ctx, np.ones(b, np.int64)
    cut = np.sort(r.randint(0, c["tokens"] + 1, b))          # the rest of the rows stays without a request
    cut[-1] = c["tokens"] - r.randint(0, 2)
    return ctx, np.diff(np.concatenate([[0], np.sort(cut)]))


# ---------------------------------------------------------------------------
# formats
# ---------------------------------------------------------------------------
def _two_to(e):
    """2^(e - 127) in fp32 from its exponent field, e from 1 to 254."""
    return (e.int() << 23).contiguous().view(torch.float32)


def _mx4(x):
    """x [..., d] fp32 -> bytes [..., d / 2] of two E2M1 codes and E8M0 codes [..., d / 32]."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    amax = b.abs().amax(-1)
    e = (((amax.view(torch.int32) + (1 << 21)) >> 23) - 2).clamp(0, 252)
    v = b.abs() * _two_to(254 - e)[..., None]
    mag = (v > 0.25).byte() + (v >= 0.75) + (v > 1.25) + (v >= 1.75) + (v > 2.5) + (v >= 3.5) + (v > 5)
    code = (mag + 8 * torch.signbit(b)).byte().reshape(x.shape)
    return code[..., 0::2] | code[..., 1::2] << 4, e.byte()


def _e2m1_pairs(dtype):
    """The two values of each byte, [256, 2]."""
    v = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=dtype, device=DEV)
    byte = torch.arange(256, device=DEV)
    return torch.stack([v[byte & 15], v[byte >> 4]], 1)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    return _prepare_attend(case, seed) if case["op"] == "attend4" else _prepare_append(case, seed)


def _int32(a):
    return torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).to(DEV)


def _table(pages_of, width, ids):
    """Rows of page ids, -1 behind each request's last page."""
    t = np.full((len(pages_of), width), -1, np.int64)
    at = 0
    for i, n in enumerate(pages_of):
        t[i, :n] = ids[at:at + n]
        at += n
    return t


def _pages8(x):
    """x [pages, heads, a, b] fp32 -> E4M3 codes and the E8M0 code of each (page, head)."""
    amax = x.abs().amax((2, 3))
    e = torch.ceil(torch.log2(amax.clamp_min(1e-30).double() / 448)).clamp(-127, 120)
    codes = (x * torch.exp2(-e).float()[:, :, None, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, (e + 127).to(torch.uint8)


def _filled_cache(gen, bits, pages, heads, page, dim):
    """A cache as a model leaves it: keys with a few strong channels, values near normal."""
    row = dim * bits // 8
    kc = torch.empty(pages, heads, page, row, dtype=torch.uint8, device=DEV)
    vc = torch.empty(pages, heads, row, page, dtype=torch.uint8, device=DEV)
    shape = (pages, heads) if bits == 8 else (pages, heads, dim // 32, page)
    ks = torch.empty(shape, dtype=torch.uint8, device=DEV)
    vs = torch.empty(shape, dtype=torch.uint8, device=DEV)
    chan = torch.exp(0.6 * torch.randn(1, heads, 1, dim, device=DEV, generator=gen))
    step = max(1, (1 << 27) // (heads * page * dim))
    for a in range(0, pages, step):
        n = min(step, pages - a)
        k = torch.randn(n, heads, page, dim, device=DEV, generator=gen) * chan
        v = torch.randn(n, heads, page, dim, device=DEV, generator=gen) * 0.5
        if bits == 8:
            kc[a:a + n], ks[a:a + n] = _pages8(k)
            vc[a:a + n], vs[a:a + n] = _pages8(v.transpose(2, 3))
        else:
            codes, scales = _mx4(k)
            kc[a:a + n], ks[a:a + n] = codes, scales.transpose(2, 3)
            codes, scales = _mx4(v)
            vc[a:a + n], vs[a:a + n] = codes.transpose(2, 3), scales.transpose(2, 3)
    return {"kc": kc, "ks": ks, "vc": vc, "vs": vs}


def _prepare_append(c, seed):
    r = np.random.RandomState(seed)
    gen = torch.Generator(DEV).manual_seed(seed)
    ctx, new = _new_lens(c, r)
    p, t = c["page"], c["tokens"]
    total = -(-(ctx + new) // p)
    # as many pages as the case can need, whatever the lengths of this seed
    ids = r.permutation(c["batch"] * (-(-c["ctx_hi"] // p) + 1) + -(-t // p) + 16)
    table = _table(total, max(1, int(total.max())), ids)
    slots, positions = np.full(t, -1, np.int64), np.full(t, -1, np.int64)
    at = 0
    for i in range(c["batch"]):
        pos = ctx[i] + np.arange(new[i])
        slots[at:at + new[i]] = table[i, pos // p] * p + pos % p
        positions[at:at + new[i]] = pos + c.get("far", 0)
        at += new[i]
    dt = torch.float32 if c["f32"] else torch.bfloat16
    # queries, keys and values as slices of one fused projection's rows, as a layer has them
    row, qrow = c["heads"] * c["dim"], c.get("q_heads", 0) * c["dim"]
    fused = torch.randn(t, qrow + 2 * row, device=DEV, generator=gen)
    fused *= torch.exp(0.6 * torch.randn(1, qrow + 2 * row, device=DEV, generator=gen))
    fused = fused.to(dt)
    s = _filled_cache(gen, c.get("bits", 4), len(ids), c["heads"], p, c["dim"])
    s.update(case=c, slots=torch.from_numpy(slots).to(DEV),
             k=fused[:, qrow:qrow + row].view(t, c["heads"], c["dim"]),
             v=fused[:, qrow + row:].view(t, c["heads"], c["dim"]))
    if c["op"] == "rotate":
        # the table of angles that a model computes once: cosines, then sines
        freq = 10000.0 ** -(torch.arange(0, c["rot"], 2, dtype=torch.float64, device=DEV) / c["rot"])
        angle = torch.arange(c["far"] + c["ctx_hi"] + t + 1, dtype=torch.float64, device=DEV)[:, None] * freq
        s.update(q=fused[:, :qrow].view(t, c["q_heads"], c["dim"]), positions=_int32(positions),
                 cos_sin=torch.cat([angle.cos(), angle.sin()], 1).float(),
                 q_out=torch.zeros(t, c["q_heads"], c["dim"], dtype=torch.bfloat16, device=DEV))
    return s


def _prepare_attend(c, seed):
    r = np.random.RandomState(seed)
    gen = torch.Generator(DEV).manual_seed(seed)
    q, kv = _attend_lens(c)
    held = -(-kv // c["page"])
    ids = r.permutation(int(held.sum()) + 8)
    s = _filled_cache(gen, 4, len(ids), c["kv_heads"], c["page"], c["dim"])
    cu = np.concatenate([[0], np.cumsum(q)])
    s.update(case=c, q=torch.randn(int(cu[-1]), c["q_heads"], c["dim"], device=DEV, generator=gen).to(torch.bfloat16),
             table=_int32(_table(held, int(held.max()) + 1, ids)), cu=_int32(cu), kv=_int32(kv), max_q=int(q.max()))
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    return {"rotate": _plain_rotate, "append4": _plain_append4, "attend4": _plain_attend4}[op](state)


def _own(s, op):
    import weight_only_quantized_quant_amd as W
    c = s["case"]
    if op == "rotate":
        q = W.wq_kv_append_rotary(s["q"], s["k"], s["v"], s["positions"], s["cos_sin"], s["slots"], s["kc"], s["ks"],
                                  s["vc"], s["vs"], interleaved=c["inter"], q_out=s["q_out"])
        return {"q": q, **_cache_values(s)}
    if op == "append4":
        W.wq_kv4_append(s["k"], s["v"], s["slots"], s["kc"], s["ks"], s["vc"], s["vs"])
        return _cache_values(s)
    out, lse = W.wq_kv4_attention(s["q"], s["kc"], s["ks"], s["vc"], s["vs"], s["table"], s["cu"], s["kv"],
                                  softcap=c["cap"], window=c["window"], max_q=s["max_q"], return_lse=True)
    return {"out": out, "lse": lse}


def _cache_values(s):
    kc, vc = s["kc"], s["vc"]
    if s["case"].get("bits", 4) == 8:
        kc, vc = kc.view(torch.float8_e4m3fn), vc.view(torch.float8_e4m3fn)
    return {"keys": kc, "key_scales": s["ks"], "values": vc, "value_scales": s["vs"]}


def _turned(x, c, cos_sin, pos):
    """x [n, heads, dim] rotated by the angles of its positions, in 64 bits."""
    x, half = x.double(), c["rot"] // 2
    cos, sin = (a[:, None] for a in cos_sin[pos].double().split(half, 1))
    a, b = (x[..., :c["rot"]:2], x[..., 1:c["rot"]:2]) if c["inter"] else x[..., :c["rot"]].split(half, -1)
    pair = (a * cos - b * sin, b * cos + a * sin)
    head = torch.stack(pair, -1).flatten(-2) if c["inter"] else torch.cat(pair, -1)
    return torch.cat([head, x[..., c["rot"]:]], -1)


def _plain_rotate(s):
    c = s["case"]
    live = (s["positions"] >= 0).nonzero()[:, 0]
    pos = s["positions"][live].long()
    s["q_out"][live] = _turned(s["q"][live], c, s["cos_sin"], pos).to(torch.bfloat16)
    k = _turned(s["k"][live], c, s["cos_sin"], pos).float()
    write = _write8 if c["bits"] == 8 else _write4
    write(s, k, s["v"][live].float(), s["slots"][live])
    return {"q": s["q_out"], **_cache_values(s)}


def _plain_append4(s):
    live = s["slots"] >= 0
    _write4(s, s["k"][live].float(), s["v"][live].float(), s["slots"][live])
    return _cache_values(s)


def _write4(s, k, v, slots):
    p = s["case"]["page"]
    page, off = slots // p, slots % p
    codes, scales = _mx4(k)
    s["kc"][page, :, off] = codes
    s["ks"][page, :, :, off] = scales
    codes, scales = _mx4(v)
    s["vc"][page, :, :, off] = codes
    s["vs"][page, :, :, off] = scales


def _write8(s, k, v, slots):
    c = s["case"]
    p = c["page"]
    page, off = slots // p, slots % p
    starts = torch.ones_like(page, dtype=torch.bool)
    starts[1:] = page[1:] != page[:-1]
    run_of = torch.cumsum(starts, 0) - 1                     # which page of the step a token goes to
    pages, first = page[starts], off[starts]
    for x, codes, scales, swap in ((k, s["kc"], s["ks"], False), (v, s["vc"], s["vs"], True)):
        amax = torch.zeros(len(pages), c["heads"], device=DEV)
        amax.scatter_reduce_(0, run_of[:, None].expand(-1, c["heads"]), x.abs().amax(2), "amax")
        frac, exp = torch.frexp(amax)                        # amax = frac 2^exp, frac in [1/2, 1)
        want = torch.where(amax > 0, (exp + 127 - 9 + (frac > 0.875)).clamp_min(0), 0)
        old = torch.where((first > 0)[:, None], scales[pages].int(), 0)
        new = torch.maximum(want, old)
        held = codes[pages]
        if swap:
            held = held.transpose(2, 3)
        keep = torch.arange(p, device=DEV)[None] < first[:, None]
        moved = held.view(torch.float8_e4m3fn).float() * torch.exp2((old - new).float())[:, :, None, None]
        moved = moved.to(torch.float8_e4m3fn).view(torch.uint8)
        held = torch.where(keep[:, None, :, None], moved, held)
        q = torch.ldexp(x, 127 - new[run_of][:, :, None]).clamp(-448, 448)
        held[run_of, :, off] = q.to(torch.float8_e4m3fn).view(torch.uint8)
        codes[pages] = held.transpose(2, 3) if swap else held
        scales[pages] = new.to(torch.uint8)


def _plain_attend4(s):
    c = s["case"]
    b, h, d, p, hq = c["batch"], c["kv_heads"], c["dim"], c["page"], c["q_heads"]
    table = s["table"].long().clamp_min(0)
    kv, cu = s["kv"].long(), s["cu"].long()
    w = table.shape[1]
    width = w * p
    pairs = _e2m1_pairs(torch.float32)
    k = pairs[s["kc"][table].int()].view(b, w, h, p, d // 32, 32)
    k = k * torch.exp2(s["ks"][table].float() - 127).transpose(3, 4)[..., None]
    k = k.permute(0, 2, 1, 3, 4, 5).reshape(b, h, width, d)
    v = pairs[s["vc"][table].int()].view(b, w, h, d // 32, 16, p, 2)
    v = v * torch.exp2(s["vs"][table].float() - 127)[:, :, :, :, None, :, None]
    v = v.permute(0, 2, 1, 5, 3, 4, 6).reshape(b, h, width, d)
    n = s["max_q"]
    row = cu[:-1, None] + torch.arange(n, device=DEV)[None]                 # [b, n]
    real = row < cu[1:, None]
    q = s["q"].float()[row.clamp_max(len(s["q"]) - 1)]                      # [b, n, hq, d]
    q = q.view(b, n, h, hq // h, d).permute(0, 2, 3, 1, 4).reshape(b, h, -1, d)
    a = torch.matmul(q, k.transpose(2, 3).contiguous()) * (1 / math.sqrt(d))
    if c["cap"]:
        a = c["cap"] * torch.tanh(a / c["cap"])
    a = a.view(b, h, hq // h, n, width)
    at = (kv - cu[1:])[:, None] + row                                       # position of each query
    j = torch.arange(width, device=DEV)
    seen = j <= at[:, :, None]
    if c["window"]:
        seen &= j > at[:, :, None] - c["window"]
    a = torch.where(seen[:, None, None], a, -math.inf)
    top = a.amax(-1, keepdim=True)
    e = torch.exp(a - torch.where(top > -math.inf, top, 0))
    total = e.sum(-1)
    o = torch.matmul(e.view(b, h, -1, width), v).view(b, h, hq // h, n, d)
    o = torch.where(total[..., None] > 0, o / total[..., None], 0)
    lse = torch.where(total > 0, torch.log(total) + top[..., 0], -math.inf)
    o = o.permute(0, 3, 1, 2, 4).reshape(b, n, hq, d)[real]
    return {"out": o.to(torch.bfloat16), "lse": lse.permute(0, 3, 1, 2).reshape(b, n, hq)[real]}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] != "attend4":
        row, t, bits = c["heads"] * c["dim"], c["tokens"], c.get("bits", 4)
        size = 4 if c["f32"] else 2
        if bits == 8:
            pages = t if c["ones"] else t / c["page"] + c["batch"]
            written = 2 * (t * row + pages * c["heads"])
        else:
            written = 2 * t * (row / 2 + row / 32)
        moved = t * (2 * row * size + 8) + written
        if c["op"] == "rotate":
            moved += t * (c["q_heads"] * c["dim"] * (size + 2) + 4 * c["rot"] + 4)
        return {"bytes": moved, "flops": 0}
    q, kv = _attend_lens(c)
    w = c["window"] or (1 << 40)
    reach = np.minimum(kv, w + q - 1)                                       # tokens that some query sees
    first = kv - q                                                          # keys before each request's first query
    pairs = sum(int(np.minimum(f + 1 + np.arange(n), w).sum()) for f, n in zip(first, q))
    size = 2 * c["kv_heads"] * int(reach.sum()) * (c["dim"] // 2 + c["dim"] // 32)
    rows = int(q.sum()) * c["q_heads"]
    return {"bytes": size + rows * (4 * c["dim"] + 4) + int(np.ceil(reach / c["page"]).sum()) * 4,
            "flops": 4 * c["dim"] * c["q_heads"] * pairs}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "append4":
        return None                                                         # whole numbers only
    s = prepare(case, seed)
    return _exact_rotate(case, s) if case["op"] == "rotate" else _exact_attend4(case, s)


def _nearest_e4m3(y):
    """Nearest E4M3 value of y (float64), ties to even, at most 448."""
    e = torch.frexp(y)[1].clamp_min(-5) - 1                                 # binary exponent, -6 for subnormals
    step = torch.exp2((e - 3).double())
    return (torch.round(y / step) * step).clamp(-448, 448)


def _exact_rotate(c, s):
    half, pos = c["rot"] // 2, s["positions"].cpu().numpy()
    at = np.nonzero(pos >= 0)[0]
    # a complex number for each pair, turned by the table's angle
    first = torch.arange(half, device=DEV) * (2 if c["inter"] else 1)
    second = first + (1 if c["inter"] else half)
    turn = torch.view_as_complex(s["cos_sin"][torch.from_numpy(pos[at]).to(DEV).long()].double().view(-1, 2, half).transpose(1, 2).contiguous())

    def turned(x):
        x = x[torch.from_numpy(at).to(DEV)].double()
        z = torch.complex(x[..., first], x[..., second]) * turn[:, None]
        x[..., first], x[..., second] = z.real, z.imag
        return x

    q = torch.zeros(s["q_out"].shape, dtype=torch.float64, device=DEV)
    q[torch.from_numpy(at).to(DEV)] = turned(s["q"])
    if c["bits"] == 4:
        return {"q": q, "keys": None, "key_scales": None, "values": None, "value_scales": None}
    p, slots = c["page"], s["slots"].cpu().numpy()[at]
    page = slots // p
    got = {"q": q}
    for name, x, codes, scales, swap in (("key", turned(s["k"]), s["kc"], s["ks"], False),
                                         ("value", s["v"][torch.from_numpy(at).to(DEV)].double(), s["vc"], s["vs"], True)):
        vals = codes.view(torch.float8_e4m3fn).double()
        new = scales.clone()
        a = 0
        while a < len(at):
            z = a
            while z < len(at) and page[z] == page[a]:
                z += 1
            pg, off = int(page[a]), int(slots[a] % p)
            t = x[a:z]                                                      # [n, heads, dim]
            amax = t.abs().amax((0, 2))
            want = torch.where(amax > 0, torch.ceil(torch.log2(amax / 448)) + 127, 0).clamp_min(0)
            old = new[pg].double() if off else torch.zeros_like(want)
            sc = torch.maximum(want, old)
            body = vals[pg].transpose(1, 2) if swap else vals[pg]           # [heads, page, dim], a view
            if off:
                body[:, :off] = _nearest_e4m3(body[:, :off] * torch.exp2(old - sc)[:, None, None])
            body[:, off:off + z - a] = _nearest_e4m3(t * torch.exp2(127 - sc)[None, :, None]).transpose(0, 1)
            new[pg] = sc.to(torch.uint8)
            a = z
        got[name + "s"] = vals
        got[name + "_scales"] = new
    return got


def _exact_attend4(c, s):
    q, kv = _attend_lens(c)
    d, group = c["dim"], c["q_heads"] // c["kv_heads"]
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=DEV)

    def values(rows, scales):
        """bytes [n, d / 2] and scales [n, d / 32] of tokens -> [n, d]."""
        x = torch.stack([rows & 15, rows >> 4], 2).flatten(1).long()
        x = grid[x & 7] * torch.where(x > 7, -1.0, 1.0)
        return x * torch.exp2(scales.double() - 127).repeat_interleave(32, 1)

    r0 = 0
    for i in range(c["batch"]):
        n, m = int(q[i]), int(kv[i])
        pages = s["table"][i, :-(-m // c["page"])].long()
        for g in range(c["kv_heads"]):
            ks, vs = (x[pages, g].transpose(1, 2).flatten(0, 1)[:m] for x in (s["ks"], s["vs"]))
            k = values(s["kc"][pages, g].flatten(0, 1)[:m], ks)
            v = values(s["vc"][pages, g].transpose(1, 2).flatten(0, 1)[:m], vs)
            for a in range(0, n, 512):
                z = min(n, a + 512)
                x = s["q"][r0 + a:r0 + z, g * group:(g + 1) * group].double()
                t = (x.reshape(-1, d) @ k.t()) / math.sqrt(d)
                if c["cap"]:
                    t = c["cap"] * torch.tanh(t / c["cap"])
                pos = (m - n + torch.arange(a, z, device=DEV)).repeat_interleave(group)[:, None]
                j = torch.arange(m, device=DEV)[None]
                dead = j > pos
                if c["window"]:
                    dead |= j <= pos - c["window"]
                t = t.masked_fill(dead, -math.inf)
                w = torch.softmax(t, 1)
                out[r0 + a:r0 + z, g * group:(g + 1) * group] = (w @ v).view(z - a, group, d)
                lse[r0 + a:r0 + z, g * group:(g + 1) * group] = torch.logsumexp(t, 1).view(z - a, group)
        r0 += n
    return {"out": out, "lse": lse}
