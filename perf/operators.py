"""Timed cases of the 4-bit paged cache and of the windowed verify attention.

Four operators of the verify step, each in a plain form of elementary torch
operations (own = False) and as a user calls the framework (own = True):

  append  quantise the new K/V rows of every sequence into 4-bit pages
          (kv_block_append_q4), then read the pages they touched back
  gather  read cached rows of 4-bit pages back as bf16 (kv_block_gather_q4)
  q4      verify attention over a 4-bit paged cache (spec_verify_attn_q4),
          with or without a sliding window and sinks
  window  verify attention with a sliding window and sinks over a bf16 or
          e4m3 paged cache (spec_verify_attn_window)

The 4-bit page. A pool is uint8 [num_blocks, H_kv, record]; the record of one
(block, kv head) holds the codes of its 16 slots, 4 bits a value, and then a
pair (scale, minimum) of f16 per slot; a value is code * scale + minimum.
  K record  slot-major: byte i of a slot's 64 code bytes holds head dim 2i in
            its low four bits and 2i + 1 in its high four; the 16-byte chunk c
            of slot s is stored at chunk c ^ ((s >> 1) & 3) of the slot
  V record  dim-major: byte i of a head dim's 8 code bytes holds slot 2i in
            its low four bits and 2i + 1 in its high four
Quantisation of a row x (all of one token and kv head, in 32 bits):
  m = f16(min x), s = f16((max x - m) / 15) raised to 2^-24, both kept within
  +-65504; code = round((x - m) / s) to the nearest even, kept within 0..15.
"""
import math
import random

import torch

own = False

BS, D = 16, 128
CODES = BS * D // 2          # code bytes of a record
RECORD = CODES + 4 * BS      # and a (scale, minimum) pair of f16 per slot
DEV = "cuda"


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # one user's next token: the append behind it, where the launch is all there is
        {"name": "append_token", "op": "append", "B": 1, "n_new": 1, "H_kv": 8, "lo": 777, "hi": 777},
        # the rows of one verify round of the 70B layer shape
        {"name": "append_verify_round", "op": "append", "B": 64, "n_new": 5, "H_kv": 8, "lo": 1024, "hi": 8192},
        # prompts entering the cache, every one of them cut at an odd place
        {"name": "append_prompts", "op": "append", "B": 16, "n_new": 2047, "H_kv": 8, "lo": 2047, "hi": 4100},
        # a short cached prefix read back before a chunk of prefill
        {"name": "gather_prefix_short", "op": "gather", "B": 3, "rows": 517, "H_kv": 8, "lo": 200, "hi": 700},
        # whole prefixes read back
        {"name": "gather_prefix_long", "op": "gather", "B": 16, "rows": 8192, "H_kv": 8, "lo": 4096, "hi": 8192},
        # one user, one token, a short context: latency
        {"name": "q4_decode_single", "op": "q4", "B": 1, "n_new": 1, "H_q": 32, "H_kv": 8, "lo": 1000, "hi": 1000, "window": 0, "sinks": 0},
        # plain decoding of a batch of short contexts
        {"name": "q4_decode_batch", "op": "q4", "B": 128, "n_new": 1, "H_q": 32, "H_kv": 8, "lo": 256, "hi": 2048, "window": 0, "sinks": 0},
        # the verify round of the 70B layer shape
        {"name": "q4_verify_70b", "op": "q4", "B": 64, "n_new": 5, "H_q": 64, "H_kv": 8, "lo": 1024, "hi": 8192, "window": 0, "sinks": 0},
        # one sequence of 128K tokens, eight query positions
        {"name": "q4_verify_128k", "op": "q4", "B": 1, "n_new": 8, "H_q": 64, "H_kv": 8, "lo": 131072, "hi": 131072, "window": 0, "sinks": 0},
        # long contexts read through a window with sinks, 4-bit pages
        {"name": "q4_window", "op": "q4", "B": 16, "n_new": 5, "H_q": 64, "H_kv": 8, "lo": 9000, "hi": 33000, "window": 4096, "sinks": 4},
        # the 70B layer shape through a window with sinks, bf16 pages
        {"name": "window_bf16_70b", "op": "window", "kv": "bf16", "B": 64, "n_new": 5, "H_q": 64, "H_kv": 8, "lo": 1024, "hi": 8192, "window": 1024, "sinks": 4},
        # many short contexts, nine query positions, a window off the page grid, e4m3 pages
        {"name": "window_fp8_batch", "op": "window", "kv": "fp8", "B": 128, "n_new": 9, "H_q": 32, "H_kv": 8, "lo": 256, "hi": 2048, "window": 500, "sinks": 17},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "gather", "q4", "q4", "window", "window"))
    if op == "append":
        H = rng.choice((1, 2, 4, 8))
        n = _log(rng, 1, 2047)
        B = max(1, min(_log(rng, 1, 128), 16 * 2047 * 8 // (n * H)))
        lo = n + _log(rng, 1, 2000) - 1
        return {"op": op, "B": B, "n_new": n, "H_kv": H, "lo": lo, "hi": lo + _log(rng, 1, 4000)}
    if op == "gather":
        H = rng.choice((1, 2, 4, 8))
        rows = _log(rng, 1, 8192)
        B = max(1, min(_log(rng, 1, 64), 12 * 8192 * 8 // (rows * H)))
        lo = max(1, rows // rng.randint(1, 4))
        return {"op": op, "B": B, "rows": rows, "H_kv": H, "lo": lo, "hi": max(lo, rows + rng.randint(-7, 300))}
    H_q, H_kv = rng.choice(((32, 8), (64, 8), (16, 2), (8, 8), (16, 1), (28, 4)))
    n = rng.randint(1, min(9, 128 * H_kv // H_q))
    hi = max(n, _log(rng, 1, 65536))
    lo = max(n, hi // rng.randint(1, 8))
    B = max(1, min(_log(rng, 1, 128), 64 * 4000 * 8 // (hi * H_kv)))
    c = {"op": op, "B": B, "n_new": n, "H_q": H_q, "H_kv": H_kv, "lo": lo, "hi": hi}
    if op == "window":
        c["kv"] = rng.choice(("bf16", "fp8"))
    windowed = op == "window" or rng.random() < 0.4
    c["window"] = _log(rng, 1, 8192) if windowed else 0
    c["sinks"] = rng.choice((0, 1, 4, 17, 64)) if windowed else 0
    return c


def _lens(case):
    """The sequences' lengths: evenly spread over lo..hi, in an order of their own. A case alone sets them."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    L = [lo + (hi - lo) * b // max(1, B - 1) for b in range(B)]
    random.Random(B * 7919 + lo).shuffle(L)
    return L


# ----------------------------------------------------------------- inputs ---

def _gen(seed, part):
    g = torch.Generator(device=DEV)
    g.manual_seed((seed * 1_000_003 + part * 7_368_787) % (2 ** 62))
    return g


def _quantise(x):
    """codes (uint8) and the (scale, minimum) pair (f16) of rows x [..., D]."""
    x = x.float()
    mn, mx = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    m = mn.clamp(-65504.0, 65504.0).half()
    s = ((mx - m.float()) / 15.0).clamp(max=65504.0).half().clamp(min=2.0 ** -24)
    c = torch.round((x - m.float()) / s.float()).clamp(0.0, 15.0).to(torch.uint8)
    return c, torch.cat((s, m), -1)


def _pair(lo, hi):
    return lo | (hi << 4)


def _chunk_order(device):
    """[slot][chunk]: where the 16-byte chunk of a slot's K codes is stored."""
    s = torch.arange(BS, device=device)[:, None]
    c = torch.arange(4, device=device)[None, :]
    return c ^ ((s >> 1) & 3)


def _k_record(c, sm):
    """codes [..., 16, D], pairs [..., 16, 2] -> records [..., RECORD]."""
    b = _pair(c[..., 0::2], c[..., 1::2]).unflatten(-1, (4, 16))
    at = _chunk_order(c.device)[..., None].expand(b.shape)
    b = torch.gather(b, -2, at)   # the exchange of chunks is its own inverse
    return torch.cat((b.flatten(-3), sm.contiguous().view(torch.uint8).flatten(-2)), -1)


def _v_record(c, sm):
    c = c.transpose(-1, -2)
    b = _pair(c[..., 0::2], c[..., 1::2])
    return torch.cat((b.flatten(-2), sm.contiguous().view(torch.uint8).flatten(-2)), -1)


def _unpair(b):
    return torch.stack((b & 15, b >> 4), -1).flatten(-2)


def _pairs_of(rec):
    return rec[..., CODES:].contiguous().view(torch.float16).unflatten(-1, (BS, 2))


def _k_codes(rec):
    b = rec[..., :CODES].unflatten(-1, (BS, 4, 16))
    at = _chunk_order(rec.device)[..., None].expand(b.shape)
    return _unpair(torch.gather(b, -2, at).flatten(-2))


def _v_codes(rec):
    return _unpair(rec[..., :CODES].unflatten(-1, (D, BS // 2))).transpose(-1, -2)


def _table(case, L, seed):
    nblk = [(x + BS - 1) // BS for x in L]
    total = sum(nblk) + 3
    g = torch.Generator()
    g.manual_seed(seed * 131 + 5)
    perm = torch.randperm(total, generator=g).to(torch.int32)
    table = torch.full((case["B"], max(nblk)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(nblk):
        table[b, :n] = perm[at:at + n]
        at += n
    return table.to(DEV), total


def _pool4(total, H_kv, seed, part, record):
    """4-bit pages that hold N(0, 1) rows."""
    pool = torch.empty(total, H_kv, RECORD, dtype=torch.uint8, device=DEV)
    g = _gen(seed, part)
    step = max(1, (1 << 27) // (H_kv * BS * D))
    for a in range(0, total, step):
        n = min(step, total - a)
        x = torch.randn((n, H_kv, BS, D), generator=g, device=DEV).bfloat16()
        pool[a:a + n] = record(*_quantise(x))
    return pool


def prepare(case, seed):
    L = _lens(case)
    H = case["H_kv"]
    table, total = _table(case, L, seed)
    s = {"op": case["op"], "table": table, "lens": torch.tensor(L, dtype=torch.int32, device=DEV)}
    if case.get("kv") == "bf16":
        for part, name in enumerate(("k", "v")):
            s[name] = torch.randn((total, H, BS, D), generator=_gen(seed, part), device=DEV).bfloat16()
        s["k_scale"] = s["v_scale"] = None
    elif case.get("kv") == "fp8":
        for part, name in enumerate(("k", "v")):
            s[name + "_scale"] = (2 + 4 * torch.rand(H, generator=_gen(seed, 20 + part), device=DEV)) / 448
            x = torch.randn((total, H, BS, D), generator=_gen(seed, part), device=DEV) / s[name + "_scale"][None, :, None, None]
            s[name] = x.clamp(-448, 448).to(torch.float8_e4m3fn)
    else:
        s["k"] = _pool4(total, H, seed, 0, _k_record)
        s["v"] = _pool4(total, H, seed, 1, _v_record)
    if case["op"] == "append":
        shape = (case["B"], case["n_new"], H, D)
        s["k_new"] = torch.randn(shape, generator=_gen(seed, 2), device=DEV).bfloat16()
        s["v_new"] = torch.randn(shape, generator=_gen(seed, 3), device=DEV).bfloat16()
        # what is read back: the new rows, and before them the rest of the first page
        s["rows"] = case["n_new"] + BS - 1
        s["start"] = (s["lens"] - s["rows"]).clamp(min=0)
    elif case["op"] == "gather":
        s["rows"] = case["rows"]
        s["start"] = torch.zeros_like(s["lens"])
    else:
        s["q"] = torch.randn((case["B"], case["n_new"], case["H_q"], D), generator=_gen(seed, 4), device=DEV).bfloat16()
        s["window"], s["sinks"] = case["window"], case["sinks"]
        s["longest"] = max(L)
    return s


# ------------------------------------------------------------ plain forms ---

def _append_plain(s):
    """The new rows quantised into their pages; the other slots of those pages stay."""
    table, lens = s["table"].long(), s["lens"].long()
    n = s["k_new"].shape[1]
    pages = (n + BS - 2) // BS + 1
    first = (lens - n) // BS
    page = first[:, None] + torch.arange(pages, device=DEV)
    used = page <= ((lens - 1) // BS)[:, None]
    block = torch.gather(table, 1, page.clamp(max=table.shape[1] - 1))
    row = (first * BS - (lens - n))[:, None] + torch.arange(pages * BS, device=DEV)   # which new row a slot takes
    new = ((row >= 0) & (row < n)).unflatten(1, (pages, BS))[:, :, None, :, None]
    row = row.clamp(0, n - 1)[:, :, None, None]
    block = block.clamp(min=0)
    for pool, x, codes_of, record in ((s["k"], s["k_new"], _k_codes, _k_record), (s["v"], s["v_new"], _v_codes, _v_record)):
        c, sm = _quantise(x)
        c = torch.gather(c, 1, row.expand(-1, -1, *c.shape[2:])).unflatten(1, (pages, BS)).transpose(2, 3)
        sm = torch.gather(sm, 1, row.expand(-1, -1, *sm.shape[2:])).unflatten(1, (pages, BS)).transpose(2, 3)
        old = pool[block]
        c = torch.where(new, c, codes_of(old))
        sm = torch.where(new, sm, _pairs_of(old))
        pool[block[used]] = record(c, sm)[used]


def _rows4(pool, codes_of, block, slot):
    """Values [B, N, H_kv, D] (f32) of 4-bit pages at (block, slot) [B, N]."""
    page, inverse = torch.unique(block, return_inverse=True)
    rec = pool[page]
    v = codes_of(rec).float()
    sm = _pairs_of(rec).float()
    v = v * sm[..., :1] + sm[..., 1:]
    return v[inverse, :, slot]


def _gather_plain(s):
    pos = s["start"].long()[:, None] + torch.arange(s["rows"], device=DEV)
    there = pos < s["lens"].long()[:, None]
    at = torch.where(there, pos, 0)
    block = torch.gather(s["table"].long(), 1, at // BS)
    return [torch.where(there[..., None, None], _rows4(s[p], f, block, at % BS), 0.0).bfloat16() for p, f in (("k", _k_codes), ("v", _v_codes))]


def _attention_plain(s):
    q, lens, table = s["q"], s["lens"].long(), s["table"].long()
    B, n, H_q, _ = q.shape
    H = s["k"].shape[1]
    W, S = s["window"], s["sinks"]
    first = lens - n
    # the keys that any query of a sequence sees: the sinks, then the window
    if W:
        begin = (first - W + 1).clamp(min=0)
        N = min(s["longest"], W + n - 1)
        pos = torch.cat((torch.arange(S, device=DEV).expand(B, S), begin[:, None] + torch.arange(N, device=DEV)), 1)
        there = torch.cat((torch.arange(S, device=DEV) < begin[:, None], pos[:, S:] < lens[:, None]), 1)
    else:
        pos = torch.arange(s["longest"], device=DEV).expand(B, -1)
        there = pos < lens[:, None]
    at = torch.where(there, pos, 0)
    block = torch.gather(table, 1, at // BS)
    slot = at % BS
    if s["op"] == "q4":
        k, v = _rows4(s["k"], _k_codes, block, slot), _rows4(s["v"], _v_codes, block, slot)
    else:
        k, v = s["k"][block, :, slot].float(), s["v"][block, :, slot].float()
        if s["k_scale"] is not None:
            k, v = k * s["k_scale"][:, None], v * s["v_scale"][:, None]
    query = first[:, None] + torch.arange(n, device=DEV)
    sees = there[:, None, :] & (pos[:, None, :] <= query[:, :, None])
    if W:
        sees &= (pos[:, None, :] > query[:, :, None] - W) | (pos[:, None, :] < S)
    G = H_q // H
    qh = q.float().view(B, n, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, n * G, D)
    x = torch.matmul(qh, k.permute(0, 2, 3, 1)) * (1 / math.sqrt(D))
    x = torch.where(sees.repeat_interleave(G, 1)[:, None], x, -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    o = torch.matmul(p / p.sum(-1, keepdim=True), v.permute(0, 2, 1, 3))
    return o.view(B, H, n, G, D).permute(0, 2, 1, 3, 4).reshape(B, n, H_q, D).to(q.dtype)


def _run_own(s):
    import speculative_verify_paged_gb300 as sv
    if s["op"] == "append":
        sv.kv_block_append_q4(s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["lens"])
    if s["op"] in ("append", "gather"):
        return list(sv.kv_block_gather_q4(s["k"], s["v"], s["table"], s["lens"], s["start"], s["rows"], D))
    if s["op"] == "q4":
        return sv.spec_verify_attn_q4(s["q"], s["k"], s["v"], s["table"], s["lens"], window=s["window"], sinks=s["sinks"])
    return sv.spec_verify_attn_window(s["q"], s["k"], s["v"], s["table"], s["lens"], s["window"], s["sinks"], k_scale=s["k_scale"], v_scale=s["v_scale"])


def run(state):
    if own:
        return _run_own(state)
    if state["op"] == "append":
        _append_plain(state)
    if state["op"] in ("append", "gather"):
        return _gather_plain(state)
    return _attention_plain(state)


# ------------------------------------------------------------------- work ---

def _visible(case, L, j):
    """How many keys query j of a sequence of length L sees."""
    p = L - case["n_new"] + j
    W = case["window"]
    if not W or p + 1 <= W:
        return p + 1
    return W + min(case["sinks"], p + 1 - W)


def work(case):
    H = case["H_kv"]
    L = _lens(case)
    if case["op"] in ("append", "gather"):
        rows = case["rows"] if case["op"] == "gather" else case["n_new"] + BS - 1
        cached = sum(min(rows, x) for x in L)
        b = cached * H * 2 * (D // 2 + 4) + case["B"] * rows * H * 2 * D * 2 + 4 * sum((min(rows, x) + BS - 1) // BS for x in L)
        f = 2 * cached * H * 2 * D
        if case["op"] == "append":
            new = case["B"] * case["n_new"] * H
            b += new * 2 * (D * 2 + D // 2 + 4)
            f += new * 2 * D * 6
        return {"bytes": b, "flops": f}
    size = {"bf16": 2 * D, "fp8": D}.get(case.get("kv"), D // 2 + 4)
    n, keys, seen = case["n_new"], 0, 0
    for x in L:
        keys += min(x, _visible(case, x, 0) + n - 1)   # read once for all the queries of a sequence
        seen += sum(_visible(case, x, j) for j in range(n))
    b = keys * H * 2 * size + 2 * case["B"] * n * case["H_q"] * D * 2 + 4 * keys // BS + 4 * case["B"]
    return {"bytes": b, "flops": 4.0 * seen * case["H_q"] * D}


# ------------------------------------------------------------------ exact ---

def _value(pool, blocks, kind):
    """Rows [n * 16, H_kv, D] in 64 bits of the listed pages, from the page's definition."""
    rec = pool[blocks].to(torch.int64)
    d, s = torch.arange(D, device=DEV), torch.arange(BS, device=DEV)
    if kind == "k":
        byte = s[:, None] * (D // 2) + (((d // 32)[None] ^ ((s // 2) % 4)[:, None]) * 16) + (d // 2)[None] % 16
        shift = (4 * (d % 2))[None].expand(BS, D)
    else:
        byte = d[None] * (BS // 2) + (s // 2)[:, None]
        shift = (4 * (s % 2))[:, None].expand(BS, D)
    code = (rec[:, :, byte] // (1 << shift)) % 16
    half = pool[blocks][..., CODES:].contiguous().view(torch.float16).double()
    v = code.double() * half[..., 0::2, None] + half[..., 1::2, None]
    return v.permute(0, 2, 1, 3).reshape(-1, pool.shape[1], D)


def _rounded_row(x):
    """What a new row becomes in the cache, in 64 bits but for the roundings that define it."""
    x = x.double()
    m = x.amin(-1, keepdim=True).clamp(-65504, 65504).half().double()
    s = ((x.amax(-1, keepdim=True) - m) / 15).clamp(max=65504).float().half().double().clamp(min=2.0 ** -24)
    return ((x - m) / s).float().double().round().clamp(0, 15) * s + m


def exact(case, seed):
    s = prepare(case, seed)
    L, H, n = _lens(case), case["H_kv"], case.get("n_new", 0)
    if case["op"] in ("append", "gather"):
        out = [torch.zeros(case["B"], s["rows"], H, D, dtype=torch.float64, device=DEV) for _ in "kv"]
        for b, x in enumerate(L):
            a = int(s["start"][b])
            e = min(x, a + s["rows"])
            blocks = s["table"][b, a // BS:(e + BS - 1) // BS].long()
            for o, kind in zip(out, "kv"):
                rows = _value(s[kind], blocks, kind)
                if case["op"] == "append":
                    rows[x - n - a // BS * BS:x - a // BS * BS] = _rounded_row(s[kind + "_new"][b])
                o[b, :e - a] = rows[a % BS:a % BS + e - a]
        return out
    G, W = case["H_q"] // H, case["window"]
    out = torch.empty(case["B"], n, case["H_q"], D, dtype=torch.float64, device=DEV)
    for b, x in enumerate(L):
        pages = torch.arange((x + BS - 1) // BS, device=DEV)
        if W:
            pages = pages[(pages * BS < case["sinks"]) | (pages * BS + BS > x - n - W + 1)]
        blocks = s["table"][b].long()[pages]
        t = (pages[:, None] * BS + torch.arange(BS, device=DEV)).flatten()
        kv = []
        for kind in "kv":
            if case["op"] == "q4":
                kv.append(_value(s[kind], blocks, kind))
            else:
                y = s[kind][blocks].double()
                if s[kind + "_scale"] is not None:
                    y = y * s[kind + "_scale"].double()[:, None, None]
                kv.append(y.permute(0, 2, 1, 3).reshape(-1, H, D))
        p = torch.arange(x - n, x, device=DEV)[:, None]
        ok = t <= p
        if W:
            ok &= (p - t < W) | (t < case["sinks"])
        for h in range(H):
            qs = s["q"][b, :, h * G:(h + 1) * G].double()
            e = torch.einsum("jgd,td->gjt", qs, kv[0][:, h]) / math.sqrt(D)
            e = torch.softmax(e.masked_fill(~ok, -math.inf), -1)
            out[b, :, h * G:(h + 1) * G] = torch.einsum("gjt,td->jgd", e, kv[1][:, h])
    return out
