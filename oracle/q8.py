"""Oracle for the 8-bit block-scaled paged cache (fp64 values, integer codes).

"KV Cache + Speculative Decoding", section 4.5 and Q9: FP8 codes with a scale,
here one for each block of tokens and kv head, set by the rows themselves.

Reading adopted (the codes are integers decided by floating point, so the
roundings are part of the definition): for the new rows of one (block, kv
head), A = their largest magnitude (NaN left out), e = the smallest integer
with A <= 448 * 2^e, kept within -32..32 (-32 for A = 0). Rows that start at
slot 0 open the block: scale = 2^e. Otherwise scale = max(old, 2^e), and where
that is larger than the old one the codes of the slots that are not written
become e4m3(code * old / new). A new element becomes e4m3(x / scale), NaN 0.
Scales are read within 2^-32 .. 2^32.

Page of one block: [H_kv][bs][d] codes, H_kv f32 scales, zeros up to a
multiple of 128 bytes.
"""

import numpy as np

from . import fp8

LO, HI = 2.0 ** -32, 2.0 ** 32


def page_bytes(H_kv, d, bs):
    return -(-(H_kv * bs * d + 4 * H_kv) // 128) * 128


def exponent(A):
    """The smallest e in -32..32 with A <= 448 * 2^e (32 where none is)."""
    for e in range(-32, 33):
        if A <= 448 * 2.0 ** e:
            return e
    return 32


def split(pool, H_kv, d, bs):
    """(codes [n, H_kv, bs, d], scales float32 [n, H_kv]) copies of pages uint8 [n, page]."""
    pool = np.ascontiguousarray(pool)
    n, at = pool.shape[0], H_kv * bs * d
    scales = np.ascontiguousarray(pool[:, at:at + 4 * H_kv]).view(np.float32).copy()
    return pool[:, :at].reshape(n, H_kv, bs, d).copy(), scales


def join(codes, scales):
    n, H, bs, d = codes.shape
    pool = np.zeros((n, page_bytes(H, d, bs)), dtype=np.uint8)
    at = H * bs * d
    pool[:, :at] = codes.reshape(n, at)
    pool[:, at:at + 4 * H] = np.ascontiguousarray(scales, dtype=np.float32).view(np.uint8)
    return pool


def read_scale(s):
    s = np.asarray(s, dtype=np.float64)
    return np.clip(np.where(np.isnan(s), LO, s), LO, HI)


def values(codes, scales):
    """fp64 values of codes [..., H, bs, d] with scales [..., H]."""
    return fp8.decode(codes) * read_scale(scales)[..., None, None]


def encode(x, scale):
    """Codes of x / scale (fp32), NaN as 0."""
    with np.errstate(over="ignore", invalid="ignore"):
        c = fp8.quantize(x, np.float32(scale))
    return np.where(np.isnan(np.asarray(x, dtype=np.float64)), 0, c).astype(np.uint8)


def append(k_cache, v_cache, k_new, v_new, block_table, seq_lens, bs=16):
    """New (k_cache, v_cache) uint8 arrays with the rows [B, n_new, H_kv, d] written."""
    out = []
    B, n_new, H, d = np.asarray(k_new).shape
    for pool, new in ((k_cache, k_new), (v_cache, v_new)):
        codes, scales = split(pool, H, d, bs)
        new = np.asarray(new, dtype=np.float32)
        for b in range(B):
            L = int(seq_lens[b])
            for page in range((L - n_new) // bs, (L - 1) // bs + 1):
                blk = int(block_table[b][page])
                slots = [s for s in range(bs) if L - n_new <= page * bs + s < L]
                for g in range(H):
                    x = np.stack([new[b, page * bs + s - (L - n_new), g] for s in slots])
                    mag = np.abs(x[~np.isnan(x)])
                    scale = 2.0 ** exponent(float(mag.max()) if mag.size else 0.0)
                    if slots[0] > 0:
                        old = float(read_scale(scales[blk, g]))
                        scale = max(old, scale)
                        if scale > old:
                            for s in range(bs):
                                if s not in slots:
                                    codes[blk, g, s] = fp8.encode(fp8.decode(codes[blk, g, s]) * (old / scale))
                    scales[blk, g] = scale
                    for s, row in zip(slots, x):
                        codes[blk, g, s] = encode(row, scale)
        out.append(join(codes, scales))
    return out[0], out[1]


def dense(pool, table_row, L, H_kv, d, bs=16):
    """Values [L, H_kv, d] (fp64) of positions 0..L-1; unused table entries give NaN rows."""
    table_row = np.asarray(table_row)[: (L + bs - 1) // bs].astype(np.int64)
    codes, scales = split(np.asarray(pool)[np.maximum(table_row, 0)], H_kv, d, bs)
    v = values(codes, scales)
    v[table_row < 0] = np.nan
    return np.moveaxis(v, 1, 2).reshape(-1, H_kv, d)[:L]
