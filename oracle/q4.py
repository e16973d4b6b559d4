"""Oracle for the 4-bit paged cache (fp64 values, integer codes).

"KV Cache + Speculative Decoding", section 4.5 and Q9: the cache holds fewer
bits per value, each row with a scale and an offset of its own.

Reading adopted (the codes are integers decided by floating point, so the
roundings are part of the definition): for a row x of one token and kv head,
in fp32,
  m = f16(min x), s = f16((max x - m) / 15) raised to 2^-24, both kept within
  +-65504; code = (x - m) / s rounded to the nearest even integer, kept within
  0..15; the value is code * s + m.
NaN elements take no part in the minimum and maximum and get code 0; a row of
nothing but NaN becomes zeros.

Record of one (block, kv head): bs * d / 2 bytes of codes, then bs pairs
(s, m) of f16. Byte by byte, written from the layout's statement:
  K: slot-major; byte i of a slot: head dim 2i low, 2i + 1 high; if d is a
     multiple of 128 the 16-byte chunk c of slot s is at c ^ ((s >> 1) & 3).
  V: dim-major; byte i of a head dim: slot 2i low, 2i + 1 high.
"""
import functools
import warnings

import numpy as np

TINY = np.float16(2.0 ** -24)


def quantize(x):
    """(codes uint8 [..., d], s float16 [...], m float16 [...]) of rows x [..., d]."""
    x = np.asarray(x, dtype=np.float32)
    with np.errstate(invalid="ignore", over="ignore"), warnings.catch_warnings():
        warnings.simplefilter("ignore", RuntimeWarning)   # rows of nothing but NaN
        mn, mx = np.nanmin(x, axis=-1), np.nanmax(x, axis=-1)
        none = np.isnan(mn)
        mn, mx = np.where(none, np.float32(0), mn), np.where(none, np.float32(0), mx)
        m = np.clip(mn, -65504, 65504).astype(np.float16)
        m32 = m.astype(np.float32)
        s = np.minimum((mx - m32) / np.float32(15), np.float32(65504)).astype(np.float16)
        s = np.maximum(s, TINY)
        c = np.rint((x - m32[..., None]) / s.astype(np.float32)[..., None])
        c = np.clip(np.where(np.isnan(c), 0, c), 0, 15).astype(np.uint8)
    return c, s, m


def values(codes, s, m):
    return codes.astype(np.float64) * s.astype(np.float64)[..., None] + m.astype(np.float64)[..., None]


@functools.lru_cache(maxsize=None)
def _places(kind, d, bs):
    """[bs][d] byte index and shift of every code in a record."""
    byte = np.empty((bs, d), dtype=np.int64)
    shift = np.empty((bs, d), dtype=np.int64)
    for slot in range(bs):
        for c in range(d):
            if kind == "k":
                chunk, rest = divmod(c // 2, 16)
                if d % 128 == 0:
                    chunk ^= (slot >> 1) & 3
                byte[slot, c], shift[slot, c] = slot * (d // 2) + chunk * 16 + rest, 4 * (c % 2)
            else:
                byte[slot, c], shift[slot, c] = c * (bs // 2) + slot // 2, 4 * (slot % 2)
    return byte, shift


def unpack(kind, rec, d, bs):
    """codes [..., bs, d], s, m [..., bs] of records uint8 [..., record]."""
    rec = np.ascontiguousarray(rec)
    byte, shift = _places(kind, d, bs)
    codes = (rec[..., byte] >> shift) & 15
    pairs = np.ascontiguousarray(rec[..., bs * d // 2:]).view(np.float16).reshape(rec.shape[:-1] + (bs, 2))
    return codes.astype(np.uint8), pairs[..., 0], pairs[..., 1]


def pack(kind, codes, s, m):
    bs, d = codes.shape[-2:]
    byte, shift = _places(kind, d, bs)
    rec = np.zeros(codes.shape[:-2] + (bs * d // 2 + 4 * bs,), dtype=np.uint8)
    for sh in (0, 4):   # every byte takes one code at each shift
        here = shift == sh
        rec[..., byte[here]] |= codes[..., here] << np.uint8(sh)
    pairs = np.stack((s, m), axis=-1).astype(np.float16)
    rec[..., bs * d // 2:] = np.ascontiguousarray(pairs).view(np.uint8).reshape(rec.shape[:-1] + (4 * bs,))
    return rec


def append(k_cache, v_cache, k_new, v_new, block_table, seq_lens, bs=16):
    """New (k_cache, v_cache) uint8 arrays with the rows [B, n_new, H_kv, d] written."""
    out = [np.array(k_cache), np.array(v_cache)]
    B, n_new, H_kv, d = np.asarray(k_new).shape
    for pool, kind, new in zip(out, "kv", (k_new, v_new)):
        codes, s, m = quantize(new)
        for b in range(B):
            for j in range(n_new):
                pos = int(seq_lens[b]) - n_new + j
                blk, slot = int(block_table[b][pos // bs]), pos % bs
                for g in range(H_kv):
                    c0, s0, m0 = unpack(kind, pool[blk, g], d, bs)
                    c0[slot], s0, m0 = codes[b, j, g], s0.copy(), m0.copy()
                    s0[slot], m0[slot] = s[b, j, g], m[b, j, g]
                    pool[blk, g] = pack(kind, c0, s0, m0)
    return out[0], out[1]


def dense(kind, pool, table_row, L, d, bs=16):
    """Values [L, H_kv, d] (fp64) of positions 0..L-1; unused table entries give NaN rows."""
    table_row = np.asarray(table_row)[: (L + bs - 1) // bs].astype(np.int64)
    codes, s, m = unpack(kind, np.asarray(pool)[np.maximum(table_row, 0)], d, bs)
    v = values(codes, s, m)
    v[table_row < 0] = np.nan
    return np.moveaxis(v, 1, 2).reshape(-1, v.shape[1], d)[:L]
