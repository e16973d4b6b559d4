"""Timed cases of rotary positions and of the 8-bit block-scaled paged cache.

Four operators of the verify step, each in a plain form of elementary torch
operations (own = False) and as a user calls the framework (own = True):

  rope    rotary positions of the new queries and keys (spec_rope)
  append  quantise the new K/V rows of every sequence into 8-bit pages
          (kv_block_append_q8), then read the pages they touched back
  gather  read cached rows of 8-bit pages back as bf16 (kv_block_gather_q8)
  q8      verify attention over an 8-bit paged cache (spec_verify_attn_q8),
          with or without a sliding window and sinks

Rotary positions. Pair i of the r rotated dims (from dim `offset` on) of a row
at position p turns by the angle p * w_i, times m:
  (a, b) -> m (a cos - b sin, b cos + a sin)
half layout: a, b = dims i and i + r / 2; interleaved: dims 2i and 2i + 1. The
other dims stay. w_i = theta^(-2i / r), changed by the scaling for long contexts.

The 8-bit page. A pool is uint8 [num_blocks, page]; a page holds the e4m3 codes
of its block, [H_kv][16][128], then one f32 scale per kv head, and is padded to
a multiple of 128 bytes; a value is code * scale. Quantisation of the new rows
of a (block, kv head): A = their largest magnitude, e = the smallest integer
with A <= 448 * 2^e, kept within -32..32 (-32 for A = 0). Where the rows start
at slot 0 the block's scale becomes 2^e; else it becomes the larger of 2^e and
the old scale, and the codes that were there are rounded anew if it grew.
"""
import math
import random

import torch

own = False

BS, D = 16, 128
DEV = "cuda"


# ------------------------------------------------------------------ cases ---

def _rope_case(name, B, n_new, H_q, H_kv, lo, hi, d=D, r=D, offset=0, pairs="half", theta=500000.0, scaling="none", dtype="bf16"):
    return {"name": name, "op": "rope", "B": B, "n_new": n_new, "H_q": H_q, "H_kv": H_kv, "lo": lo, "hi": hi, "d": d, "r": r,
            "offset": offset, "pairs": pairs, "theta": theta, "scaling": scaling, "dtype": dtype}


def _attn_case(name, B, n_new, H_q, H_kv, lo, hi, window=0, sinks=0):
    return {"name": name, "op": "q8", "B": B, "n_new": n_new, "H_q": H_q, "H_kv": H_kv, "lo": lo, "hi": hi, "window": window,
            "sinks": sinks}


def listed():
    return [
        # one user's next token at an ordinary position: the launch is all there is
        _rope_case("rope_token", 1, 1, 64, 8, 777, 777, scaling="bands"),
        # a verify round of absorbed latent queries, 64 rotated dims behind 512, contexts stretched to 128K
        _rope_case("rope_latent_round", 32, 5, 128, 1, 20000, 131072, d=576, r=64, offset=512, pairs="interleaved", theta=10000.0,
                   scaling="yarn"),
        # prompts of an odd length, half of each head rotated
        _rope_case("rope_prompts", 16, 2047, 64, 8, 2047, 4100, r=64, theta=10000.0, scaling="linear"),
        # the rows of one verify round of the 70B layer shape, into blocks that hold rows already
        {"name": "append_verify_round", "op": "append", "B": 64, "n_new": 5, "H_kv": 8, "lo": 1024, "hi": 8192},
        # prompts entering the cache, every one of them cut at an odd place
        {"name": "append_prompts", "op": "append", "B": 16, "n_new": 2047, "H_kv": 8, "lo": 2047, "hi": 4100},
        # a short cached prefix read back before a chunk of prefill
        {"name": "gather_prefix_short", "op": "gather", "B": 3, "rows": 517, "H_kv": 8, "lo": 200, "hi": 700},
        # whole prefixes read back
        {"name": "gather_prefix_long", "op": "gather", "B": 16, "rows": 8192, "H_kv": 8, "lo": 4096, "hi": 8192},
        # one user, one token, a short context: latency
        _attn_case("q8_decode_single", 1, 1, 32, 8, 1000, 1000),
        # plain decoding of a batch of short contexts
        _attn_case("q8_decode_batch", 128, 1, 32, 8, 256, 2048),
        # the verify round of the 70B layer shape
        _attn_case("q8_verify_70b", 64, 5, 64, 8, 1024, 8192),
        # one sequence of 128K tokens, eight query positions
        _attn_case("q8_verify_128k", 1, 8, 64, 8, 131072, 131072),
        # long contexts read through a window with sinks
        _attn_case("q8_window", 16, 5, 64, 8, 9000, 33000, window=4096, sinks=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope", "rope", "append", "gather", "q8", "q8"))
    if op == "rope":
        d, offset, H_q, H_kv = rng.choice(((128, 0, 64, 8), (128, 0, 32, 8), (64, 0, 32, 8), (256, 0, 16, 1), (96, 0, 28, 4), (576, 512, 128, 1), (576, 512, 16, 1)))
        r = d - offset if offset or rng.random() < 0.5 else 2 * rng.randint(1, d // 2)
        n = _log(rng, 1, 2047)
        dtype = rng.choice(("bf16", "bf16", "f32"))
        most = 16 * 2047 * 72 * 128 // (n * (H_q + H_kv) * d * (2 if dtype == "f32" else 1))
        c = _rope_case(None, max(1, min(_log(rng, 1, 128), most)), n, H_q, H_kv, n, n, d=d, r=r, offset=offset,
                       pairs=rng.choice(("half", "interleaved")), theta=rng.choice((10000.0, 500000.0, 1000000.0)),
                       scaling=rng.choice(("none", "linear", "bands", "yarn")), dtype=dtype)
        c["lo"] = n + _log(rng, 1, 100000) - 1
        c["hi"] = c["lo"] + _log(rng, 1, 30000)
        c.pop("name")
        return c
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
    windowed = rng.random() < 0.4
    c = _attn_case(None, B, n, H_q, H_kv, lo, hi, window=_log(rng, 1, 8192) if windowed else 0,
                   sinks=rng.choice((0, 1, 4, 17, 64)) if windowed else 0)
    c.pop("name")
    return c


def _lens(case):
    """The sequences' lengths: evenly spread over lo..hi, in an order of their own. A case alone sets them."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    L = [lo + (hi - lo) * b // max(1, B - 1) for b in range(B)]
    random.Random(B * 7919 + lo).shuffle(L)
    return L


# How positions are stretched: w_i as a function of theta^(-2i / r).
SCALINGS = {
    "none": {},
    # every frequency divided
    "linear": {"kind": "linear", "factor": 4.0},
    # long wavelengths divided, short ones kept, a ramp between
    "bands": {"kind": "llama3", "factor": 8.0, "low_freq_factor": 1.0, "high_freq_factor": 4.0, "original_length": 8192},
    # a ramp over the pairs' index, and a factor on cos and sin
    "yarn": {"kind": "yarn", "factor": 32.0, "beta_fast": 32.0, "beta_slow": 1.0, "original_length": 4096},
}


def _frequencies(case):
    """(w_0 .. w_(r/2 - 1), m) in double precision."""
    r, theta, s = case["r"], case["theta"], SCALINGS[case["scaling"]]
    w = [theta ** (-2.0 * i / r) for i in range(r // 2)]
    kind = s.get("kind")
    if kind is None:
        return w, 1.0
    f = s["factor"]
    if kind == "linear":
        return [x / f for x in w], 1.0
    n = s["original_length"]
    if kind == "llama3":
        lo, hi = s["low_freq_factor"], s["high_freq_factor"]
        out = []
        for x in w:
            turns = n * x / (2 * math.pi)   # over the original context
            keep = min(1.0, max(0.0, (turns - lo) / (hi - lo)))
            out.append(x * keep + x / f * (1 - keep))
        return out, 1.0

    def pair_of(turns):   # the pair that makes so many turns over the original context
        return r * math.log(n / (turns * 2 * math.pi)) / (2 * math.log(theta))
    lo = max(math.floor(pair_of(s["beta_fast"])), 0)
    hi = min(math.ceil(pair_of(s["beta_slow"])), r - 1)
    if hi == lo:
        hi += 0.001
    out = []
    for i, x in enumerate(w):
        ramp = min(1.0, max(0.0, (i - lo) / (hi - lo)))
        out.append(x / f * ramp + x * (1 - ramp))
    return out, 0.1 * math.log(f) + 1.0


# ----------------------------------------------------------------- inputs ---

def _gen(seed, part):
    g = torch.Generator(device=DEV)
    g.manual_seed((seed * 1_000_003 + part * 7_368_787) % (2 ** 62))
    return g


def _rows(shape, g, key):
    """N(0, 1) rows [..., D] whose size differs from token to token; keys have a few large channels."""
    x = torch.randn(shape, generator=g, device=DEV)
    x *= torch.exp(0.4 * torch.randn((*shape[:-1], 1), generator=g, device=DEV))
    if key:
        x[..., 5::31] *= 6.0
    return x.bfloat16()


def _exponent(x):
    """e of the rows x [..., rows, D] that share it."""
    a = x.abs().amax((-1, -2))
    m, e = torch.frexp(a)   # a = m 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
    e = torch.where(m > 0.875, e - 8, e - 9)
    return torch.where(a == 0, -32, e.clamp(-32, 32))


def _power(e):
    """2^e (f32) for whole e within -126..127."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _codes(x, e):
    """e4m3 codes (uint8) of x / 2^e."""
    y = (x * _power(-e)).clamp(-448.0, 448.0)
    return y.to(torch.float8_e4m3fn).view(torch.uint8)


def _page_bytes(H):
    return (H * (BS * D + 4) + 127) // 128 * 128


def _split(pool, H):
    """Views of a pool: codes [num_blocks, H, 16, D] (uint8) and scales [num_blocks, H] (f32)."""
    n, at = pool.shape[0], H * BS * D
    return pool[:, :at].view(n, H, BS, D), pool[:, at:at + 4 * H].view(torch.float32)


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


def _pool(total, H, seed, part):
    """8-bit pages that hold rows."""
    pool = torch.zeros(total, _page_bytes(H), dtype=torch.uint8, device=DEV)
    codes, scales = _split(pool, H)
    g = _gen(seed, part)
    step = max(1, (1 << 26) // (H * BS * D))
    for a in range(0, total, step):
        x = _rows((min(step, total - a), H, BS, D), g, part == 0).float()
        e = _exponent(x)
        codes[a:a + step] = _codes(x, e[..., None, None])
        scales[a:a + step] = _power(e)
    return pool


def prepare(case, seed):
    L = _lens(case)
    s = {"op": case["op"], "case": case, "lens": torch.tensor(L, dtype=torch.int32, device=DEV)}
    if case["op"] == "rope":
        t = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        for part, (name, H) in enumerate((("q", case["H_q"]), ("k", case["H_kv"]))):
            s[name] = torch.randn((case["B"], case["n_new"], H, case["d"]), generator=_gen(seed, part), device=DEV).to(t)
        s["rope"] = None   # the handle, made by the first call
        return s
    H = case["H_kv"]
    s["table"], total = _table(case, L, seed)
    s["k"], s["v"] = _pool(total, H, seed, 0), _pool(total, H, seed, 1)
    if case["op"] == "append":
        shape = (case["B"], case["n_new"], H, D)
        s["k_new"] = _rows(shape, _gen(seed, 2), True)
        s["v_new"] = _rows(shape, _gen(seed, 3), False)
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

def _rope_plain(s):
    case = s["case"]
    w, m = _frequencies(case)
    w = torch.tensor(w, dtype=torch.float64, device=DEV)
    pos = s["lens"].double()[:, None] - case["n_new"] + torch.arange(case["n_new"], device=DEV)
    angle = pos[..., None] * w                       # (32 bits lose the angles of far positions)
    cos = (torch.cos(angle) * m).float()[:, :, None]
    sin = (torch.sin(angle) * m).float()[:, :, None]
    at, r = case["offset"], case["r"]
    out = []
    for x in (s["q"], s["k"]):
        y = x.clone()
        rot = x[..., at:at + r].float()
        if case["pairs"] == "half":
            a, b = rot[..., :r // 2], rot[..., r // 2:]
            y[..., at:at + r // 2] = (a * cos - b * sin).to(x.dtype)
            y[..., at + r // 2:at + r] = (b * cos + a * sin).to(x.dtype)
        else:
            a, b = rot[..., 0::2], rot[..., 1::2]
            y[..., at:at + r:2] = (a * cos - b * sin).to(x.dtype)
            y[..., at + 1:at + r:2] = (b * cos + a * sin).to(x.dtype)
        out.append(y)
    return out


def _append_plain(s):
    """The new rows quantised into their pages; the other slots of those pages keep their values."""
    table, lens = s["table"].long(), s["lens"].long()
    n, H = s["k_new"].shape[1:3]
    pages = (n + BS - 2) // BS + 1
    first = (lens - n) // BS
    page = first[:, None] + torch.arange(pages, device=DEV)
    used = page <= ((lens - 1) // BS)[:, None]
    block = torch.gather(table, 1, page.clamp(max=table.shape[1] - 1)).clamp(min=0)[used]
    row = ((first * BS - (lens - n))[:, None] + torch.arange(pages * BS, device=DEV)).unflatten(1, (pages, BS))   # which new row a slot takes
    new = ((row >= 0) & (row < n))[used][:, None, :, None]
    opens = (row[..., 0] >= 0)[used][:, None]         # the block's first slot is written
    seq = torch.arange(table.shape[0], device=DEV)[:, None, None].expand_as(row)
    row, seq = row.clamp(0, n - 1)[used], seq[used]
    for pool, x in ((s["k"], s["k_new"]), (s["v"], s["v_new"])):
        codes, scales = _split(pool, H)
        x = torch.where(new, x[seq, row].float().transpose(1, 2), 0.0)
        e = _exponent(x)
        old = scales[block]
        fresh = _power(e)
        scale = torch.where(opens, fresh, torch.maximum(old, fresh))
        e = torch.frexp(scale)[1] - 1
        was = codes[block]
        moved = _codes(was.view(torch.float8_e4m3fn).float() * old[..., None, None], e[..., None, None])
        keep = torch.where((opens | (scale == old))[..., None, None], was, moved)
        codes[block] = torch.where(new, _codes(x, e[..., None, None]), keep)
        scales[block] = scale


def _values(pool, H, block, slot):
    """Values [B, N, H, D] (f32) of 8-bit pages at (block, slot) [B, N]."""
    codes, scales = _split(pool, H)
    return codes[block, :, slot].view(torch.float8_e4m3fn).float() * scales[block][..., None]


def _gather_plain(s):
    H = s["case"]["H_kv"]
    pos = s["start"].long()[:, None] + torch.arange(s["rows"], device=DEV)
    there = pos < s["lens"].long()[:, None]
    at = torch.where(there, pos, 0)
    block = torch.gather(s["table"].long(), 1, at // BS)
    return [torch.where(there[..., None, None], _values(s[p], H, block, at % BS), 0.0).bfloat16() for p in ("k", "v")]


def _attention_plain(s):
    q, lens, table = s["q"], s["lens"].long(), s["table"].long()
    B, n, H_q, _ = q.shape
    H = s["case"]["H_kv"]
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
    k, v = _values(s["k"], H, block, at % BS), _values(s["v"], H, block, at % BS)
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
    if s["op"] == "rope":
        if s["rope"] is None:
            c = s["case"]
            s["rope"] = sv.Rope(c["r"], theta=c["theta"], interleaved=c["pairs"] == "interleaved", offset=c["offset"],
                                scaling=SCALINGS[c["scaling"]] or None)
        return list(sv.spec_rope(s["q"], s["k"], s["rope"], seq_lens=s["lens"]))
    if s["op"] == "append":
        sv.kv_block_append_q8(s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["lens"])
    if s["op"] in ("append", "gather"):
        return list(sv.kv_block_gather_q8(s["k"], s["v"], s["table"], s["lens"], s["start"], s["rows"], D))
    return sv.spec_verify_attn_q8(s["q"], s["k"], s["v"], s["table"], s["lens"], window=s["window"], sinks=s["sinks"])


def run(state):
    if own:
        return _run_own(state)
    if state["op"] == "rope":
        return _rope_plain(state)
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
    if case["op"] == "rope":
        rows = case["B"] * case["n_new"] * (case["H_q"] + case["H_kv"])
        return {"bytes": 2 * rows * case["d"] * (4 if case["dtype"] == "f32" else 2) + 4 * case["B"], "flops": 3 * rows * case["r"]}
    H = case["H_kv"]
    L = _lens(case)
    if case["op"] in ("append", "gather"):
        rows = case["rows"] if case["op"] == "gather" else case["n_new"] + BS - 1
        cached = sum(min(rows, x) for x in L)
        pages = sum((min(rows, x) + BS - 1) // BS for x in L)
        b = cached * H * 2 * D + pages * (8 * H + 4) + case["B"] * rows * H * 2 * D * 2
        f = cached * H * 2 * D
        if case["op"] == "append":
            new = case["B"] * case["n_new"] * H
            b += new * 2 * (D * 2 + D)
            f += new * 2 * D * 3
        return {"bytes": b, "flops": f}
    n, keys, seen = case["n_new"], 0, 0
    for x in L:
        keys += min(x, _visible(case, x, 0) + n - 1)   # read once for all the queries of a sequence
        seen += sum(_visible(case, x, j) for j in range(n))
    b = keys * H * 2 * D + keys // BS * (8 * H + 4) + 2 * case["B"] * n * case["H_q"] * D * 2 + 4 * case["B"]
    return {"bytes": b, "flops": 4.0 * seen * case["H_q"] * D}


# ------------------------------------------------------------------ exact ---

def _code_values():
    """The 256 values of e4m3 by its definition: a sign, four exponent bits (bias 7), three fraction bits."""
    out = []
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        x = f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        out.append(-x if c >> 7 else x)
    return torch.tensor(out, dtype=torch.float64, device=DEV)


def _stored(pool, blocks, H):
    """(values [n, H, 16, D], scales [n, H]) of the listed pages in 64 bits."""
    raw = pool[blocks]
    scale = raw[:, H * BS * D:H * (BS * D + 4)].contiguous().view(torch.float32).double().view(-1, H)
    v = _code_values()[raw[:, :H * BS * D].long()].view(-1, H, BS, D)
    return v * scale[..., None, None], scale


def _two_to(e):
    """2^e in 64 bits for whole e within -64..64."""
    return torch.tensor([2.0 ** k for k in range(-64, 65)], dtype=torch.float64, device=DEV)[e.long() + 64]


def _to_e4m3(x):
    """x in 64 bits to the nearest e4m3 value, ties to the even one, the largest 448."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    step = _two_to(e - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _append_exact(case, s):
    out = [torch.zeros(case["B"], s["rows"], case["H_kv"], D, dtype=torch.float64, device=DEV) for _ in "kv"]
    H, n = case["H_kv"], case["n_new"]
    for b, x in enumerate(_lens(case)):
        a = int(s["start"][b])
        p0, p1 = a // BS, (x + BS - 1) // BS
        blocks = s["table"][b, p0:p1].long()
        for o, kind in zip(out, "kv"):
            values, old = _stored(s[kind], blocks, H)
            new = torch.zeros((p1 - p0) * BS, H, D, dtype=torch.float64, device=DEV)
            new[x - n - p0 * BS:x - p0 * BS] = s[kind + "_new"][b].double()
            new = new.view(-1, BS, H, D).transpose(1, 2)
            at = torch.arange(p0 * BS, p1 * BS, device=DEV).view(-1, 1, BS, 1)
            fresh = (at >= x - n) & (at < x)
            touched = fresh.any(2)[..., 0]
            opens = fresh[:, :, 0, 0]
            largest = 448 * _two_to(torch.arange(-32, 32, device=DEV))
            scale = _two_to((new.abs().amax((2, 3))[..., None] > largest).sum(-1) - 32)
            scale = torch.where(opens, scale, torch.maximum(scale, old))
            scale = torch.where(touched, scale, old)
            grown = (touched & ~opens & (scale > old))[..., None, None]
            scale = scale[..., None, None]
            values = torch.where(grown, _to_e4m3(values / scale) * scale, values)
            rows = torch.where(fresh, _to_e4m3(new / scale) * scale, values).transpose(1, 2).reshape(-1, H, D)
            end = min(x, a + s["rows"])
            o[b, :end - a] = rows[a - p0 * BS:end - p0 * BS]
    return out


def _rope_exact(case, s):
    w, m = _frequencies(case)
    out = []
    for name in "qk":
        x = s[name].double()
        c = x[..., case["offset"]:case["offset"] + case["r"]]
        if case["pairs"] == "half":
            c = c.unflatten(-1, (2, -1)).transpose(-1, -2)
        else:
            c = c.unflatten(-1, (-1, 2))
        c = torch.view_as_complex(c.contiguous())
        for b, L in enumerate(_lens(case)):
            for i, f in enumerate(w):
                a = f * torch.arange(L - case["n_new"], L, dtype=torch.float64, device=DEV)
                c[b, ..., i] *= torch.polar(torch.full_like(a, m), a)[:, None]
        c = torch.view_as_real(c)
        if case["pairs"] == "half":
            c = c.transpose(-1, -2)
        x[..., case["offset"]:case["offset"] + case["r"]] = c.flatten(-2)
        out.append(x)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _rope_exact(case, s)
    if case["op"] == "append":
        return _append_exact(case, s)
    L, H = _lens(case), case["H_kv"]
    if case["op"] == "gather":
        out = [torch.zeros(case["B"], s["rows"], H, D, dtype=torch.float64, device=DEV) for _ in "kv"]
        for b, x in enumerate(L):
            e = min(x, s["rows"])
            for o, kind in zip(out, "kv"):
                v = _stored(s[kind], s["table"][b, :(e + BS - 1) // BS].long(), H)[0]
                o[b, :e] = v.transpose(1, 2).reshape(-1, H, D)[:e]
        return out
    n, G, W = case["n_new"], case["H_q"] // H, case["window"]
    out = torch.empty(case["B"], n, case["H_q"], D, dtype=torch.float64, device=DEV)
    for b, x in enumerate(L):
        pages = torch.arange((x + BS - 1) // BS, device=DEV)
        if W:
            pages = pages[(pages * BS < case["sinks"]) | (pages * BS + BS > x - n - W + 1)]
        blocks = s["table"][b].long()[pages]
        t = (pages[:, None] * BS + torch.arange(BS, device=DEV)).flatten()
        k, v = (_stored(s[kind], blocks, H)[0].transpose(0, 1).reshape(H, -1, D) for kind in "kv")
        p = torch.arange(x - n, x, device=DEV)[:, None]
        ok = t <= p
        if W:
            ok &= (p - t < W) | (t < case["sinks"])
        for h in range(H):
            qs = s["q"][b, :, h * G:(h + 1) * G].double()
            e = torch.einsum("jgd,td->gjt", qs, k[h]) / math.sqrt(D)
            e = torch.softmax(e.masked_fill(~ok, -math.inf), -1)
            out[b, :, h * G:(h + 1) * G] = torch.einsum("gjt,td->jgd", e, v[h])
    return out
