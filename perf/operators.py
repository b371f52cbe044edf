"""Measured cases of the 8-bit paged key/value cache: its block tables, its
append, and the attention that reads it.

A cache page holds `page` tokens.  Keys are E4M3 codes [pages, kv_heads, page,
dim], values E4M3 codes [pages, kv_heads, dim, page] (transposed, the order
in which the second product reads them), and each (page, head) has one E8M0
scale for its keys and one for its values.  A block table row lists the pages
of one request.

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
        # One scheduler step of a full server: every request gets one token, a
        # few of them a new page.
        {"name": "blocks_step", "op": "blocks", "batch": 256, "tokens": 256, "ones": True, "ctx_hi": 32768, "page": 64,
         "width": 520},
        # The first step of a handful of ragged prompts with small pages: the
        # tables are built from the lengths, and the token arrays have spare rows.
        {"name": "blocks_prompts", "op": "blocks", "batch": 7, "tokens": 16384, "ones": False, "ctx_hi": 0, "page": 16,
         "width": 1024},
        # One decode step's new keys and values: 64 requests, one token each,
        # most of them in the middle of a page.
        {"name": "append_step", "op": "append", "batch": 64, "tokens": 64, "ones": True, "ctx_hi": 500, "heads": 8,
         "dim": 128, "page": 64, "f32": False},
        # Whole prompts written at once.
        {"name": "append_prompts", "op": "append", "batch": 6, "tokens": 8192, "ones": False, "ctx_hi": 0, "heads": 8,
         "dim": 128, "page": 64, "f32": False},
        # Chunks that begin and end inside pages: an odd number of tokens,
        # three heads of 64, pages of 16, inputs in 32 bits.
        {"name": "append_odd", "op": "append", "batch": 11, "tokens": 1037, "ones": False, "ctx_hi": 300, "heads": 3,
         "dim": 64, "page": 16, "f32": True},
        # One request decoding alone: latency.
        {"name": "attend_single", "op": "attend", "batch": 1, "ones": 1, "q_lo": 1, "q_hi": 1, "kv_lo": 1000,
         "kv_hi": 1000, "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "cap": 0.0, "window": 0, "lens": 1},
        # A decode batch at ordinary contexts.
        {"name": "attend_batch", "op": "attend", "batch": 64, "ones": 64, "q_lo": 1, "q_hi": 1, "kv_lo": 2048,
         "kv_hi": 8192, "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "cap": 0.0, "window": 0, "lens": 2},
        # One very long context beside short ones, large pages.
        {"name": "attend_long", "op": "attend", "batch": 5, "ones": 5, "q_lo": 1, "q_hi": 1, "kv_lo": 200,
         "kv_hi": 131072, "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 128, "cap": 0.0, "window": 0, "lens": 3},
        # As many key heads as query heads, heads of 64, capped scores, a
        # sliding window, pages of 16, an odd batch.
        {"name": "attend_window", "op": "attend", "batch": 33, "ones": 33, "q_lo": 1, "q_hi": 1, "kv_lo": 1,
         "kv_hi": 5000, "q_heads": 16, "kv_heads": 16, "dim": 64, "page": 16, "cap": 30.0, "window": 1000, "lens": 4},
        # A few drafted tokens per request checked at once, five query heads
        # to a key head.
        {"name": "attend_verify", "op": "attend", "batch": 24, "ones": 3, "q_lo": 2, "q_hi": 7, "kv_lo": 500,
         "kv_hi": 6000, "q_heads": 40, "kv_heads": 8, "dim": 128, "page": 32, "cap": 0.0, "window": 0, "lens": 5},
        # Whole prompts against the cache they were just written to.
        {"name": "attend_prompts", "op": "attend", "batch": 3, "ones": 0, "q_lo": 1500, "q_hi": 4096, "kv_lo": 1500,
         "kv_hi": 4096, "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "cap": 0.0, "window": 0, "lens": 6},
        # A mixed step: chunks of long prompts beside decoding requests, with
        # capped scores.
        {"name": "attend_chunks", "op": "attend", "batch": 6, "ones": 4, "q_lo": 700, "q_hi": 1024, "kv_lo": 4000,
         "kv_hi": 16000, "q_heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "cap": 50.0, "window": 0, "lens": 7},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["blocks", "append", "append", "attend", "attend", "attend", "attend"])
    page = rng.choice([16, 32, 64, 128])
    if kind == "blocks":
        batch = _log_int(rng, 1, 256)
        if rng.random() < 0.5:
            ctx = _log_int(rng, 100, 8192)
            return {"op": "blocks", "batch": batch, "tokens": batch + rng.choice([0, 0, 5]), "ones": True,
                    "ctx_hi": ctx, "page": page, "width": ctx // page + 3}
        tokens = _log_int(rng, batch * 2, 16384)
        return {"op": "blocks", "batch": batch, "tokens": tokens, "ones": False, "ctx_hi": rng.choice([0, 200]),
                "page": page, "width": (tokens + 200) // page + 2}
    if kind == "append":
        ones = rng.random() < 0.4
        batch = _log_int(rng, 1, 128) if ones else _log_int(rng, 1, 12)
        tokens = batch if ones else _log_int(rng, batch * 8, 8192)
        return {"op": "append", "batch": batch, "tokens": tokens, "ones": ones, "ctx_hi": rng.choice([0, 100, 500]),
                "heads": rng.choice([1, 2, 3, 8]), "dim": rng.choice([64, 128]), "page": page,
                "f32": rng.random() < 0.25}
    top = {"bytes": 0, "flops": 0}
    for c in listed():
        if c["op"] == "attend":
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
        c = {"op": "attend", "batch": batch, "ones": batch if shape == "step" else rng.randint(0, batch // 2),
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
    """Lengths before the step and new tokens of each request for the table and append cases."""
    b = c["batch"]
    ctx = np.exp(r.uniform(0, math.log(c["ctx_hi"]), b)).astype(np.int64) if c["ctx_hi"] else np.zeros(b, np.int64)
    if c["ones"]:
        return ctx, np.ones(b, np.int64)
    cut = np.sort(r.randint(0, c["tokens"] + 1, b))          # the rest of the rows stays without a request
    cut[-1] = c["tokens"] - r.randint(0, 2)
    return ctx, np.diff(np.concatenate([[0], np.sort(cut)]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    return {"blocks": _prepare_blocks, "append": _prepare_append, "attend": _prepare_attend}[case["op"]](case, seed)


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


def _prepare_blocks(c, seed):
    r = np.random.RandomState(seed)
    ctx, new = _new_lens(c, r)
    p = c["page"]
    held = -(-ctx // p)
    need = -(-(ctx + new) // p) - held
    ids = r.permutation(int(held.sum() + need.sum()) + 64)
    return {"case": c, "ctx": _int32(ctx), "new": _int32(new), "table": _int32(_table(held, c["width"], ids)),
            "free": _int32(ids[held.sum():]), "cursor": _int32(np.zeros(1))}


def _pages_e4m3(x):
    """x [pages, heads, a, b] fp32 -> E4M3 codes and the E8M0 code of each (page, head)."""
    amax = x.abs().amax((2, 3))
    e = torch.ceil(torch.log2(amax.clamp_min(1e-30).double() / 448)).clamp(-127, 120)
    codes = (x * torch.exp2(-e).float()[:, :, None, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, (e + 127).to(torch.uint8)


def _filled_cache(gen, pages, heads, page, dim):
    """A cache as a model leaves it: keys with a few strong channels, values near normal."""
    kc = torch.empty(pages, heads, page, dim, dtype=torch.uint8, device=DEV)
    vc = torch.empty(pages, heads, dim, page, dtype=torch.uint8, device=DEV)
    ks = torch.empty(pages, heads, dtype=torch.uint8, device=DEV)
    vs = torch.empty(pages, heads, dtype=torch.uint8, device=DEV)
    chan = torch.exp(0.6 * torch.randn(1, heads, 1, dim, device=DEV, generator=gen))
    step = max(1, (1 << 27) // (heads * page * dim))
    for a in range(0, pages, step):
        n = min(step, pages - a)
        x = torch.randn(n, heads, page, dim, device=DEV, generator=gen) * chan
        kc[a:a + n], ks[a:a + n] = _pages_e4m3(x)
        x = torch.randn(n, heads, dim, page, device=DEV, generator=gen) * 0.5
        vc[a:a + n], vs[a:a + n] = _pages_e4m3(x)
    return {"kc": kc, "ks": ks, "vc": vc, "vs": vs}


def _prepare_append(c, seed):
    r = np.random.RandomState(seed)
    gen = torch.Generator(DEV).manual_seed(seed)
    ctx, new = _new_lens(c, r)
    p = c["page"]
    total = -(-(ctx + new) // p)
    # as many pages as the case can need, whatever the lengths of this seed
    ids = r.permutation(c["batch"] * (-(-c["ctx_hi"] // p) + 1) + -(-c["tokens"] // p) + 16)
    table = _table(total, max(1, int(total.max())), ids)
    slots = np.full(c["tokens"], -1, np.int64)
    at = 0
    for i in range(c["batch"]):
        pos = ctx[i] + np.arange(new[i])
        slots[at:at + new[i]] = table[i, pos // p] * p + pos % p
        at += new[i]
    dt = torch.float32 if c["f32"] else torch.bfloat16
    # keys and values as slices of one fused projection's rows, as a layer has them
    row = c["heads"] * c["dim"]
    fused = torch.randn(c["tokens"], 2 * row, device=DEV, generator=gen)
    fused *= torch.exp(0.6 * torch.randn(1, 2 * row, device=DEV, generator=gen))
    fused = fused.to(dt)
    s = _filled_cache(gen, len(ids), c["heads"], p, c["dim"])
    s.update(case=c, slots=torch.from_numpy(slots).to(DEV),
             k=fused[:, :row].view(c["tokens"], c["heads"], c["dim"]),
             v=fused[:, row:].view(c["tokens"], c["heads"], c["dim"]))
    return s


def _prepare_attend(c, seed):
    r = np.random.RandomState(seed)
    gen = torch.Generator(DEV).manual_seed(seed)
    q, kv = _attend_lens(c)
    held = -(-kv // c["page"])
    ids = r.permutation(int(held.sum()) + 8)
    s = _filled_cache(gen, len(ids), c["kv_heads"], c["page"], c["dim"])
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
    return {"blocks": _plain_blocks, "append": _plain_append, "attend": _plain_attend}[op](state)


def _own(s, op):
    import weight_only_quantized_quant_amd as W
    c = s["case"]
    if op == "blocks":
        got = W.wq_kv_blocks(s["ctx"], s["new"], s["free"], s["table"], c["page"], c["tokens"], cursor=s["cursor"])
        slots, positions, cu_new, kv_lens, cursor = got
        return {"table": s["table"], "slots": slots, "positions": positions, "cu": cu_new, "kv": kv_lens,
                "cursor": cursor}
    if op == "append":
        W.wq_kv_append(s["k"], s["v"], s["slots"], s["kc"], s["ks"], s["vc"], s["vs"])
        return _cache_values(s)
    out, lse = W.wq_kv_attention(s["q"], s["kc"], s["ks"], s["vc"], s["vs"], s["table"], s["cu"], s["kv"],
                                 softcap=c["cap"], window=c["window"], max_q=s["max_q"], return_lse=True)
    return {"out": out, "lse": lse}


def _cache_values(s):
    return {"keys": s["kc"].view(torch.float8_e4m3fn), "key_scales": s["ks"],
            "values": s["vc"].view(torch.float8_e4m3fn), "value_scales": s["vs"]}


def _plain_blocks(s):
    c, ctx, new, table = s["case"], s["ctx"].long(), s["new"].long(), s["table"]
    p, t, width = c["page"], c["tokens"], c["width"]
    held, total = (ctx + p - 1) // p, (ctx + new + p - 1) // p
    need = torch.where(total <= width, total - held, 0)
    first = s["cursor"].long() + torch.cumsum(need, 0) - need
    ends = torch.cumsum(new, 0)
    ok = (total <= width) & ((need == 0) | (first + need <= s["free"].numel())) & (ends <= t)
    cols = torch.arange(width, device=DEV)[None]
    fresh = (cols >= held[:, None]) & (cols < total[:, None]) & ok[:, None]
    at = (first[:, None] + cols - held[:, None]).clamp(0, s["free"].numel() - 1)
    table.copy_(torch.where(fresh, s["free"][at], table))
    tok = torch.arange(t, device=DEV)
    seq = torch.searchsorted(ends, tok, right=True).clamp_max(len(ctx) - 1)
    live = (tok < ends[-1]) & ok[seq]
    pos = torch.where(live, ctx[seq] + tok - ends[seq] + new[seq], 0)
    page = table[seq, (pos // p).clamp_max(width - 1)].long()
    live &= page >= 0
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), ends]).clamp_max(t)
    used = s["cursor"].long() + torch.where(ok, need, 0).sum()
    return {"table": table, "slots": torch.where(live, page * p + pos % p, -1),
            "positions": torch.where(live, pos, -1).int(), "cu": cu.int(),
            "kv": torch.where(ok, ctx + new, ctx).int(), "cursor": torch.cat([used, (~ok).sum()[None]]).int()}


def _plain_append(s):
    c = s["case"]
    p = c["page"]
    live = s["slots"] >= 0
    slots = s["slots"][live]
    page, off = slots // p, slots % p
    starts = torch.ones_like(live[live])
    starts[1:] = page[1:] != page[:-1]
    run_of = torch.cumsum(starts, 0) - 1                     # which page of the step a token goes to
    pages, first = page[starts], off[starts]
    for x, codes, scales, swap in ((s["k"], s["kc"], s["ks"], False), (s["v"], s["vc"], s["vs"], True)):
        x = x[live].float()
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
    return _cache_values(s)


def _plain_attend(s):
    c = s["case"]
    b, h, d, p, hq = c["batch"], c["kv_heads"], c["dim"], c["page"], c["q_heads"]
    table = s["table"].long().clamp_min(0)
    kv, cu = s["kv"].long(), s["cu"].long()
    width = table.shape[1] * p

    def values(codes, scales):
        x = codes[table].view(torch.float8_e4m3fn).float()
        return x * torch.exp2(scales[table].float() - 127)[..., None, None]

    k = values(s["kc"], s["ks"]).permute(0, 2, 1, 3, 4).reshape(b, h, width, d)
    v = values(s["vc"], s["vs"]).permute(0, 2, 1, 4, 3).reshape(b, h, width, d)
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
    if c["op"] == "blocks":
        b, t = c["batch"], c["tokens"]
        pages = b * (1 / c["page"]) if c["ones"] else t / c["page"] + b / 2
        return {"bytes": b * (8 + 8) + t * 12 + pages * 8, "flops": 0}
    if c["op"] == "append":
        row = c["heads"] * c["dim"]
        pages = c["tokens"] if c["ones"] else c["tokens"] / c["page"] + c["batch"]
        return {"bytes": c["tokens"] * (2 * row * ((4 if c["f32"] else 2) + 1) + 8) + pages * c["heads"] * 4, "flops": 0}
    q, kv = _attend_lens(c)
    w = c["window"] or (1 << 40)
    reach = np.minimum(kv, w + q - 1)                                       # tokens that some query sees
    first = kv - q                                                          # keys before each request's first query
    pairs = sum(int(np.minimum(f + 1 + np.arange(n), w).sum()) for f, n in zip(first, q))
    size = 2 * c["kv_heads"] * (int(reach.sum()) * c["dim"] + int(np.ceil(reach / c["page"]).sum()))
    rows = int(q.sum()) * c["q_heads"]
    return {"bytes": size + rows * (4 * c["dim"] + 4) + int(np.ceil(reach / c["page"]).sum()) * 4,
            "flops": 4 * c["dim"] * c["q_heads"] * pairs}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(case, s)
    if case["op"] == "attend":
        return _exact_attend(case, s)
    return None                                                             # whole numbers only


def _nearest_e4m3(y):
    """Nearest E4M3 value of y (float64), ties to even, at most 448."""
    e = torch.frexp(y)[1].clamp_min(-5) - 1                                 # binary exponent, -6 for subnormals
    step = torch.exp2((e - 3).double())
    return (torch.round(y / step) * step).clamp(-448, 448)


def _exact_append(c, s):
    p, slots = c["page"], s["slots"].cpu().numpy()
    at = np.nonzero(slots >= 0)[0]
    page = slots[at] // p
    got = {}
    for name, x, codes, scales, swap in (("key", s["k"], s["kc"], s["ks"], False), ("value", s["v"], s["vc"], s["vs"], True)):
        vals = codes.view(torch.float8_e4m3fn).double()
        new = scales.clone()
        a = 0
        while a < len(at):
            z = a
            while z < len(at) and page[z] == page[a]:
                z += 1
            pg, off = int(page[a]), int(slots[at[a]] % p)
            t = x[int(at[a]):int(at[a]) + z - a].double()                   # [n, heads, dim]
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


def _exact_attend(c, s):
    q, kv = _attend_lens(c)
    d, group = c["dim"], c["q_heads"] // c["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=DEV)
    r0 = 0
    for i in range(c["batch"]):
        n, m = int(q[i]), int(kv[i])
        pages = s["table"][i, :-(-m // c["page"])].long()
        for g in range(c["kv_heads"]):
            k = s["kc"][pages, g].view(torch.float8_e4m3fn).double() * torch.exp2(s["ks"][pages, g].double() - 127)[:, None, None]
            v = s["vc"][pages, g].view(torch.float8_e4m3fn).double() * torch.exp2(s["vs"][pages, g].double() - 127)[:, None, None]
            k = k.reshape(-1, d)[:m]
            v = v.transpose(1, 2).reshape(-1, d)[:m]
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
