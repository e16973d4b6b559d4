// kv_block_append_q4 and kv_block_gather_q4: the 4-bit paged cache's write and
// read-back (record layout: q4.cuh).
//
// A row x of one token and kv head becomes, in fp32 with IEEE rounding,
//   m = f16(min x), s = max(f16((max x - m) / 15), 2^-24), both kept within
//   +-65504, code = clamp(rne((x - m) / s), 0, 15).
// NaN elements are left out of the minimum and the maximum and get code 0 (a
// row of nothing but NaN becomes zeros).
// s never reaches zero, so readers may divide by it or take its logarithm;
// a constant row has every code 0 and the value m.
#include <algorithm>
#include <cstring>

#include "q4.cuh"

namespace sv {
namespace {

struct Q4AppendArgs {
  const void *src[2];   // K, V rows [B][n_new][H_kv][d]
  uint8_t *cache[2];
  const int32_t *block_table, *seq_lens;
  int max_blocks, n_new, H_kv, bs, num_blocks;
  int64_t block_stride, head_stride;   // bytes
  int32_t *status;
};

constexpr int kQaWarps = 4;
constexpr int kQaRows = 2;   // rows of K, and of V, that a group of lanes takes at a time

// Eight consecutive elements of a row as floats; `vec`: 16-byte aligned.
template <typename T>
__device__ __forceinline__ void load8(const T *p, bool vec, T (&x)[8]) {
  if (vec) {
#pragma unroll
    for (int k = 0; k < (int)sizeof(T) / 2; ++k)
      reinterpret_cast<uint4 *>(x)[k] = reinterpret_cast<const uint4 *>(p)[k];
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = p[k];
  }
}

// Eight elements of no row: NaN, which takes no part in anything.
template <typename T>
__device__ __forceinline__ void no_row(T (&x)[8]) {
#pragma unroll
  for (int k = 0; k < (int)sizeof(T) * 2; ++k)
    reinterpret_cast<uint32_t *>(x)[k] = sizeof(T) == 2 ? 0x7FC07FC0u : 0x7FC00000u;
}

// Smallest and largest of the 8 LPR elements of a group of lanes, NaN left out
// (no more than NaN: NaN or mn > mx).
template <int LPR>
__device__ __forceinline__ void extremes(const __nv_bfloat16 (&x)[8], float &mn, float &mx) {
  // exact in bf16; (min, -max) travel together
  const __nv_bfloat162 *p = reinterpret_cast<const __nv_bfloat162 *>(x);
  const __nv_bfloat162 lo = __hmin2(__hmin2(p[0], p[1]), __hmin2(p[2], p[3]));
  const __nv_bfloat162 hi = __hmax2(__hmax2(p[0], p[1]), __hmax2(p[2], p[3]));
  uint32_t a, b;
  memcpy(&a, &lo, 4);
  memcpy(&b, &hi, 4);
  b ^= 0x80008000u;
  const uint32_t c = __byte_perm(a, b, 0x5410), d = __byte_perm(a, b, 0x7632);
  __nv_bfloat162 v, o;
  memcpy(&v, &c, 4);
  memcpy(&o, &d, 4);
  v = __hmin2(v, o);
#pragma unroll
  for (int k = LPR / 2; k > 0; k >>= 1) {
    memcpy(&a, &v, 4);
    a = __shfl_xor_sync(0xffffffffu, a, k);
    memcpy(&o, &a, 4);
    v = __hmin2(v, o);
  }
  mn = __low2float(v);
  mx = -__high2float(v);
}
template <int LPR>
__device__ __forceinline__ void extremes(const float (&x)[8], float &mn, float &mx) {
  mn = INFINITY;   // (fminf and fmaxf leave NaN out)
  mx = -INFINITY;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    mn = fminf(mn, x[k]);
    mx = fmaxf(mx, x[k]);
  }
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) {
    mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  }
}

// x: eight words of eight 4-bit values, word j nibble i. Afterwards nibbles of
// equal place lie in equal bytes: bits 0-3 of byte k of x[i] and x[i + 1] (i
// even) are nibble i of words 2k and 2k + 1, bits 4-7 their nibble i + 1.
__device__ __forceinline__ void transpose8(uint32_t (&x)[8]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {   // halves, across a distance of four words
    const uint32_t a = x[k], b = x[k + 4];
    x[k] = __byte_perm(a, b, 0x5410);
    x[k + 4] = __byte_perm(a, b, 0x7632);
  }
#pragma unroll
  for (int h = 0; h < 8; h += 4)
#pragma unroll
    for (int k = 0; k < 2; ++k) {   // bytes, across two
      const uint32_t a = x[h + k], b = x[h + k + 2];
      x[h + k] = __byte_perm(a, b, 0x6240);
      x[h + k + 2] = __byte_perm(a, b, 0x7351);
    }
}

// One CTA per (block that new rows land in, kv head, sequence). A group of
// lanes takes a row, eight elements a lane: minimum, maximum and a word of
// eight codes, which for K is a word of the record and for V goes to shared
// memory, where the CTA turns words along the head dim into words along the
// slots. Words of a V record that also hold codes of other slots are read and
// merged; no other CTA of the call touches the record.
// The quotient (x - m) / s is first taken as 15 times ((x - m) times 1 / (15 s),
// kept within 0..1). The reciprocal's error is 2^-23, the product's 2^-24 and the
// IEEE quotient's 2^-24 relative, so the two differ by less than 15 x 2^-22; only
// where a value lies within 2^-16 of the middle between two codes is the division
// done.
// Measured: 2 x 16 x 2047 bf16 rows of 8 heads of 128 (170 MB to move, 25 us at
// the measured bandwidth) take 57 us (f32 rows: 64): bound by instruction issue
// (82 % of the slots, some 200 warp instructions for two rows). One lane per row
// works out its scale; with all lanes of a row doing so it took 8 us more. Twelve
// CTAs an SM (40 registers) against nine: 2 us.
template <typename TIn, int NE>
__global__ void __launch_bounds__(32 * kQaWarps, sizeof(TIn) == 2 ? 12 : 8) q4_append_kernel(const __grid_constant__ Q4AppendArgs a, bool vec) {
  constexpr int d = 32 * NE, W = d / 8;                              // words of a row
  constexpr int LPR = NE == 1 ? 4 : NE == 2 ? 8 : NE <= 4 ? 16 : 32;  // lanes of a row (those past W idle)
  constexpr int kGroups = 32 * kQaWarps / LPR;
  constexpr float kMagic = 12582912.f;                               // 1.5 x 2^23: adding it rounds to an integer
  extern __shared__ __align__(16) uint32_t qa_smem[];
  uint32_t *words = qa_smem;                // [bs][W] of V, eight head dims each
  uint32_t *image = qa_smem + a.bs * W;     // the V record's codes
  pdl_trigger();
  const int g = blockIdx.y, b = blockIdx.z;
  const int group = threadIdx.x / LPR, li = threadIdx.x % LPR;
  const int bs = a.bs;
  const int L = a.seq_lens[b];
  // (every CTA waits, so that this grid ends after the one before it)
  if (L < a.n_new || L > a.max_blocks * bs) {
    pdl_wait();
    if (threadIdx.x == 0 && g == 0 && blockIdx.x == 0) atomic_or_status(a.status, SV_DEV_BAD_SEQ_LEN);
    return;
  }
  const int first = L - a.n_new;
  const int page = first / bs + (int)blockIdx.x;
  const int s0 = max(first - page * bs, 0), s1 = min(L - page * bs, bs);   // slots written
  if (s0 >= s1) {
    pdl_wait();
    return;
  }
  const int phys = a.block_table[(int64_t)b * a.max_blocks + page];
  const int nr = s1 - s0;
  const int64_t row_stride = (int64_t)a.H_kv * d;
  const int64_t src0 = (((int64_t)b * a.n_new + (page * bs + s0 - first)) * a.H_kv + g) * d + li * 8;
  const int64_t rec0 = (int64_t)phys * a.block_stride + (int64_t)g * a.head_stride;
  const bool on = li < W;
  // the new rows may be what the kernel before reads back (q4_gather_kernel),
  // and the pools may still be read by it
  pdl_wait();
  if (phys < 0 || phys >= a.num_blocks) {
    if (threadIdx.x == 0) atomic_or_status(a.status, SV_DEV_BAD_BLOCK);
    return;
  }
  for (int i0 = 0; i0 < nr; i0 += kQaRows * kGroups) {
    // (rows 0 .. kQaRows - 1 are of K, the others of V)
    alignas(16) TIn xr[2 * kQaRows][8];
#pragma unroll
    for (int u = 0; u < 2 * kQaRows; ++u) {
      const int i = i0 + u % kQaRows * kGroups + group;
      no_row(xr[u]);
      if (i < nr && on) load8(static_cast<const TIn *>(a.src[u / kQaRows]) + src0 + i * row_stride, vec, xr[u]);
    }
    // lane u of the group works out row u's pair
    float mn = 0.f, mx = 0.f;
#pragma unroll
    for (int u = 0; u < 2 * kQaRows; ++u) {
      float lo, hi;
      extremes<LPR>(xr[u], lo, hi);
      if (li == u) {
        mn = lo;
        mx = hi;
      }
    }
    if (!(mn <= mx)) mn = mx = 0.f;   // nothing but NaN
    const __half mh = __float2half_rn(fminf(fmaxf(mn, -65504.f), 65504.f));
    const __half sh = __hmax(__float2half_rn(fminf(__fdiv_rn(__fsub_rn(mx, __half2float(mh)), 15.f), 65504.f)),
                             __ushort_as_half(1));
    const uint32_t own = (uint32_t)__half_as_ushort(sh) | ((uint32_t)__half_as_ushort(mh) << 16);
    float own_inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(own_inv) : "f"(15.f * __half2float(sh)));
    if (li < 2 * kQaRows) {
      const int i = i0 + li % kQaRows * kGroups + group;
      if (i < nr)
        *reinterpret_cast<uint32_t *>((li < kQaRows ? a.cache[0] : a.cache[1]) + rec0 + q4_code_bytes(d, bs) + 4 * (s0 + i)) = own;
    }
#pragma unroll
    for (int u = 0; u < 2 * kQaRows; ++u) {
      const int i = i0 + u % kQaRows * kGroups + group, slot = s0 + i;
      const uint32_t pair = __shfl_sync(0xffffffffu, own, u, LPR);
      const float inv = __shfl_sync(0xffffffffu, own_inv, u, LPR);
      const float m = __half2float(__ushort_as_half((unsigned short)(pair >> 16)));
      uint32_t w = 0;
      float near = 0.f;   // distance from a code, the largest of the eight
      const float2 m2 = make_float2(-m, -m), magic2 = make_float2(kMagic, kMagic), less2 = make_float2(-kMagic, -kMagic);
#pragma unroll
      for (int k = 6; k >= 0; k -= 2) {
        const float2 y = __fadd2_rn(make_float2(to_f32(xr[u][k]), to_f32(xr[u][k + 1])), m2);
        const float2 t = make_float2(__saturatef(y.x * inv), __saturatef(y.y * inv));   // (NaN: 0)
        const float2 r = __ffma2_rn(t, make_float2(15.f, 15.f), magic2);
        const float2 c = __fadd2_rn(r, less2);
        const float2 e = __ffma2_rn(t, make_float2(-15.f, -15.f), c);
        near = fmaxf(fmaxf(near, fabsf(e.x)), fabsf(e.y));
        w = (w << 4) + __float_as_uint(r.y);   // (the bits of kMagic come off below)
        w = (w << 4) + __float_as_uint(r.x);
      }
      w -= 0x4B400000u * 0x11111111u;
      if (near > 0.5f - 0x1p-16f) {
        const float s = __half2float(__ushort_as_half((unsigned short)pair));
        w = 0;
#pragma unroll
        for (int k = 7; k >= 0; --k)
          w = (w << 4) + (uint32_t)(int)fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(to_f32(xr[u][k]), m), s)), 0.f), 15.f);
      }
      if (i < nr && on) {
        if (u >= kQaRows) words[slot * W + li] = w;
        else *reinterpret_cast<uint32_t *>(a.cache[0] + rec0 + q4_k_byte(slot, 8 * li, d)) = w;
      }
    }
  }
  __syncthreads();
  // V: eight head dims by eight slots a thread
  const int wpd = bs / 8;   // words of a head dim
  for (int i = threadIdx.x; i < W * wpd; i += 32 * kQaWarps) {
    const int o = i % W, t0 = 8 * (i / W);
    uint32_t x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = t0 + k >= s0 && t0 + k < s1 ? words[(t0 + k) * W + o] : 0;
    transpose8(x);
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
      image[(8 * o + k) * wpd + i / W] = (x[k] & 0x0F0F0F0Fu) | ((x[k + 1] & 0x0F0F0F0Fu) << 4);
      image[(8 * o + k + 1) * wpd + i / W] = ((x[k] >> 4) & 0x0F0F0F0Fu) | (x[k + 1] & 0xF0F0F0F0u);
    }
  }
  __syncthreads();
  uint8_t *rec = a.cache[1] + rec0;
  if (nr == bs) {
    for (int i = threadIdx.x; i < d * bs / 32; i += 32 * kQaWarps)
      reinterpret_cast<uint4 *>(rec)[i] = reinterpret_cast<const uint4 *>(image)[i];
    return;
  }
  for (int i = threadIdx.x; i < d * wpd; i += 32 * kQaWarps) {
    const int t0 = 8 * (i % wpd);
    if (t0 + 8 <= s0 || t0 >= s1) continue;
    const int lo = max(s0 - t0, 0), hi = min(s1 - t0, 8);
    const uint32_t mask = (0xFFFFFFFFu << (4 * lo)) & (0xFFFFFFFFu >> (32 - 4 * hi));
    uint32_t *p = reinterpret_cast<uint32_t *>(rec) + i;
    *p = mask == 0xFFFFFFFFu ? image[i] : (image[i] & mask) | (*p & ~mask);
  }
}

struct Q4GatherArgs {
  const uint8_t *cache[2];
  void *out[2];   // [B][n_rows][H_kv][d]
  const int32_t *block_table, *seq_lens, *start;
  int max_blocks, n_rows, H_kv, bs, num_blocks, pages;   // pages: blocks that n_rows rows can touch
  int64_t block_stride, head_stride;   // bytes
  int32_t *status;
};

// Eight codes (even elements in the bytes of e, odd ones in those of o) as
// code * scale + minimum to eight consecutive elements of a row.
template <typename TO>
__device__ __forceinline__ void write8(TO *dst, bool vec, uint32_t e, uint32_t o, float s, float m) {
  float v[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {   // (a byte under the exponent of 2^23 is 2^23 + the byte)
    v[2 * k] = fmaf(__uint_as_float(__byte_perm(e, 0x4B000000u, 0x7540 + k)) - 8388608.f, s, m);
    v[2 * k + 1] = fmaf(__uint_as_float(__byte_perm(o, 0x4B000000u, 0x7540 + k)) - 8388608.f, s, m);
  }
  if (vec) {
    uint4 w[sizeof(TO) / 2];
    if constexpr (sizeof(TO) == 4) {
      memcpy(w, v, sizeof(w));
    } else {
      __nv_bfloat162 h[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) h[k] = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
      memcpy(w, h, sizeof(w));
    }
#pragma unroll
    for (int k = 0; k < (int)sizeof(TO) / 2; ++k) reinterpret_cast<uint4 *>(dst)[k] = w[k];
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if constexpr (sizeof(TO) == 4) dst[k] = v[k];
      else dst[k] = __float2bfloat16_rn(v[k]);
    }
  }
}

// A warp takes one block of one kv head: first the K record, a word (eight head
// dims of a slot) a lane and step, then the V record, eight head dims by eight
// slots a lane, turned in registers. Rows are written eight elements at a time,
// a row's lanes side by side. Rows outside the sequence, and those of a block
// with a number out of range, are written as zeros. Bound by HBM: 16 x 8192 rows
// of 8 heads of 128 (643 MB) take 99 us, 6.5 TB/s (a thread per value: 906 us);
// as f32 rows (1.22 GB) 236 us.
constexpr int kQgWarps = 8;
template <typename TO, int NE>
__global__ void __launch_bounds__(32 * kQgWarps) q4_gather_kernel(const __grid_constant__ Q4GatherArgs a, bool vec) {
  constexpr int d = 32 * NE, W = d / 8, kStep = 4;
  pdl_trigger();
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * kQgWarps + (threadIdx.x >> 5);
  const int g = (int)(unit % a.H_kv);
  const int64_t p = unit / a.H_kv;
  const int bs = a.bs;
  const int L = a.seq_lens[b], start = a.start[b];
  pdl_wait();
  if (p >= a.pages) return;
  const bool len_ok = L >= 0 && L <= a.max_blocks * bs;
  if (!len_ok && lane == 0 && unit == 0) atomic_or_status(a.status, SV_DEV_BAD_SEQ_LEN);
  const int64_t page = (start >= 0 ? start / bs : -((bs - 1 - (int64_t)start) / bs)) + p;
  const int64_t i0 = page * bs - start;   // output row of slot 0
  const int r0 = (int)max((int64_t)0, -i0), r1 = (int)min((int64_t)bs, a.n_rows - i0);   // slots to write
  if (r0 >= r1) return;
  int held = len_ok && page >= 0 ? (int)min((int64_t)bs, max((int64_t)0, L - page * bs)) : 0;   // slots that hold rows
  int phys = 0;
  if (held > 0) {
    phys = a.block_table[(int64_t)b * a.max_blocks + page];
    if (phys < 0 || phys >= a.num_blocks) {
      if (lane == 0) atomic_or_status(a.status, SV_DEV_BAD_BLOCK);
      phys = held = 0;
    }
  }
  const int64_t rec = (int64_t)phys * a.block_stride + (int64_t)g * a.head_stride;
  const int64_t stride = (int64_t)a.H_kv * d;
  const int64_t at = ((int64_t)b * a.n_rows + i0) * stride + (int64_t)g * d;   // of slot 0
  const int code_bytes = q4_code_bytes(d, bs);
  const uint8_t *kr = a.cache[0] + rec, *vr = a.cache[1] + rec;
  const int steps = bs * NE / 8;
  for (int k0 = 0; k0 < steps; k0 += kStep) {
    uint32_t w[kStep], pr[kStep];
#pragma unroll
    for (int u = 0; u < kStep; ++u) {
      const int i = (k0 + u) * 32 + lane, slot = i / W;
      w[u] = pr[u] = 0;
      if (k0 + u < steps && slot < held) {
        w[u] = *reinterpret_cast<const uint32_t *>(kr + q4_k_byte(slot, 8 * (i % W), d));
        pr[u] = *reinterpret_cast<const uint32_t *>(kr + code_bytes + 4 * slot);
      }
    }
#pragma unroll
    for (int u = 0; u < kStep; ++u) {
      const int i = (k0 + u) * 32 + lane, slot = i / W;
      if (k0 + u >= steps || slot < r0 || slot >= r1) continue;
      const float2 sm = __half22float2(*reinterpret_cast<const __half2 *>(&pr[u]));
      write8(static_cast<TO *>(a.out[0]) + at + slot * stride + 8 * (i % W), vec, w[u] & 0x0F0F0F0Fu,
             (w[u] >> 4) & 0x0F0F0F0Fu, sm.x, sm.y);
    }
  }
  const int wpd = bs / 8;
  for (int i = lane; i < W * wpd; i += 32) {
    const int o = i % W, t = i / W;
    uint32_t x[8], pr[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      x[k] = pr[k] = 0;
      if (8 * t < held) x[k] = reinterpret_cast<const uint32_t *>(vr)[(8 * o + k) * wpd + t];
      if (8 * t + k < held) pr[k] = reinterpret_cast<const uint32_t *>(vr + code_bytes)[8 * t + k];
    }
    transpose8(x);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int slot = 8 * t + k;
      if (slot < r0 || slot >= r1) continue;
      const float2 sm = __half22float2(*reinterpret_cast<const __half2 *>(&pr[k]));
      const uint32_t e = k & 1 ? x[k - 1] >> 4 : x[k], od = k & 1 ? x[k] >> 4 : x[k + 1];
      write8(static_cast<TO *>(a.out[1]) + at + slot * stride + 8 * o, vec, e & 0x0F0F0F0Fu, od & 0x0F0F0F0Fu, sm.x, sm.y);
    }
  }
}

template <typename TIn, int NE>
sv_status launch_append_q4(const Q4AppendArgs &a, int B, cudaStream_t s) {
  const int pages = (a.n_new + a.bs - 2) / a.bs + 1;
  const bool vec = aligned(a.src[0], 16) && aligned(a.src[1], 16);
  launch_k(q4_append_kernel<TIn, NE>, dim3(pages, a.H_kv, B), dim3(32 * kQaWarps), (size_t)a.bs * 32 * NE, s, 1, a,
           vec);
  return check_launch("kv_block_append_q4 launch");
}

template <typename TIn>
sv_status launch_append_q4_d(const Q4AppendArgs &a, int d, int B, cudaStream_t s) {
  switch (d / 32) {
    case 1: return launch_append_q4<TIn, 1>(a, B, s);
    case 2: return launch_append_q4<TIn, 2>(a, B, s);
    case 3: return launch_append_q4<TIn, 3>(a, B, s);
    case 4: return launch_append_q4<TIn, 4>(a, B, s);
    case 5: return launch_append_q4<TIn, 5>(a, B, s);
    case 6: return launch_append_q4<TIn, 6>(a, B, s);
    case 7: return launch_append_q4<TIn, 7>(a, B, s);
    default: return launch_append_q4<TIn, 8>(a, B, s);
  }
}

template <typename TO, int NE>
sv_status launch_gather_q4(const Q4GatherArgs &a, int B, cudaStream_t s) {
  const bool vec = aligned(a.out[0], 16) && aligned(a.out[1], 16);
  const int64_t ctas = ((int64_t)a.pages * a.H_kv + kQgWarps - 1) / kQgWarps;
  if (ctas >= (1ll << 31)) return fail(SV_ERR_UNSUPPORTED, "kv_block_gather_q4: too many rows");
  launch_k(q4_gather_kernel<TO, NE>, dim3((unsigned)ctas, B), dim3(32 * kQgWarps), 0, s, 1, a, vec);
  return check_launch("kv_block_gather_q4 launch");
}

template <typename TO>
sv_status launch_gather_q4_d(const Q4GatherArgs &a, int d, int B, cudaStream_t s) {
  switch (d / 32) {
    case 1: return launch_gather_q4<TO, 1>(a, B, s);
    case 2: return launch_gather_q4<TO, 2>(a, B, s);
    case 3: return launch_gather_q4<TO, 3>(a, B, s);
    case 4: return launch_gather_q4<TO, 4>(a, B, s);
    case 5: return launch_gather_q4<TO, 5>(a, B, s);
    case 6: return launch_gather_q4<TO, 6>(a, B, s);
    case 7: return launch_gather_q4<TO, 7>(a, B, s);
    default: return launch_gather_q4<TO, 8>(a, B, s);
  }
}

}  // namespace

// What the 4-bit entry points share: sizes, alignment and the record strides.
sv_status q4_check(const char *what, const void *k_cache, const void *v_cache, const sv_kv_layout *layout, int H_kv,
                   int d_head, int block_size, int64_t *block_stride, int64_t *head_stride) {
  if (d_head % 32 || d_head > 256 || block_size % 8 || block_size > 64)
    return fail(SV_ERR_UNSUPPORTED,
                "%s: 4-bit pools take d_head a multiple of 32 up to 256 and block_size a multiple of 8 up to 64", what);
  const int64_t rec = q4_record_bytes(d_head, block_size);
  if (layout) {
    *block_stride = layout->block_stride;
    *head_stride = layout->head_stride;
    if (layout->slot_stride != 0 || *head_stride < rec || *block_stride < rec || *head_stride % 16 || *block_stride % 16)
      return fail(SV_ERR_INVALID_ARG,
                  "%s: the layout of a 4-bit pool has record strides in bytes (multiples of 16, at least %lld) and "
                  "slot_stride 0",
                  what, (long long)rec);
  } else {
    *head_stride = rec;
    *block_stride = rec * H_kv;
  }
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16))
    return fail(SV_ERR_INVALID_ARG, "%s: 4-bit pools must be 16-byte aligned", what);
  return SV_OK;
}

}  // namespace sv

extern "C" size_t sv_q4_record_bytes(int d_head, int block_size) {
  if (d_head < 32 || d_head % 32 || d_head > 256 || block_size < 8 || block_size % 8 || block_size > 64) return 0;
  return (size_t)sv::q4_record_bytes(d_head, block_size);
}

extern "C" sv_status kv_block_append_q4(const void *k_new, const void *v_new, sv_dtype new_dtype, void *k_cache,
                                        void *v_cache, const sv_kv_layout *layout, const int32_t *block_table,
                                        int max_blocks_per_seq, const int32_t *seq_lens, int B, int n_new, int H_kv,
                                        int d_head, int block_size, int num_blocks, int32_t *dev_status,
                                        sv_stream_t stream) {
  using namespace sv;
  if (!k_new || !v_new || !k_cache || !v_cache || !block_table || !seq_lens)
    return fail(SV_ERR_INVALID_ARG, "kv_block_append_q4: null pointer argument");
  if (B < 0 || n_new < 1 || H_kv < 1 || d_head < 1 || block_size < 1 || num_blocks < 1 || max_blocks_per_seq < 1)
    return fail(SV_ERR_INVALID_ARG, "kv_block_append_q4: bad sizes");
  if (new_dtype != SV_F32 && new_dtype != SV_BF16)
    return fail(SV_ERR_UNSUPPORTED, "kv_block_append_q4: new rows must be f32 or bf16");
  if (B > 65535 || H_kv > 65535) return fail(SV_ERR_UNSUPPORTED, "kv_block_append_q4: B or H_kv too large");
  if (!capacity_ok(max_blocks_per_seq, block_size))
    return fail(SV_ERR_UNSUPPORTED, "kv_block_append_q4: max_blocks_per_seq * block_size must be below 2^30");
  Q4AppendArgs a = {};
  const sv_status rc = q4_check("kv_block_append_q4", k_cache, v_cache, layout, H_kv, d_head, block_size,
                                &a.block_stride, &a.head_stride);
  if (rc != SV_OK) return rc;
  if (B == 0) return ok();
  a.src[0] = k_new; a.src[1] = v_new;
  a.cache[0] = static_cast<uint8_t *>(k_cache); a.cache[1] = static_cast<uint8_t *>(v_cache);
  a.block_table = block_table; a.seq_lens = seq_lens; a.max_blocks = max_blocks_per_seq; a.n_new = n_new;
  a.H_kv = H_kv; a.bs = block_size; a.num_blocks = num_blocks; a.status = dev_status;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (new_dtype == SV_F32) return launch_append_q4_d<float>(a, d_head, B, s);
  return launch_append_q4_d<__nv_bfloat16>(a, d_head, B, s);
}

extern "C" sv_status kv_block_gather_q4(const void *k_cache, const void *v_cache, const sv_kv_layout *layout,
                                        const int32_t *block_table, int max_blocks_per_seq, const int32_t *seq_lens,
                                        const int32_t *start, int B, int n_rows, int H_kv, int d_head, int block_size,
                                        int num_blocks, void *k_out, void *v_out, sv_dtype out_dtype,
                                        int32_t *dev_status, sv_stream_t stream) {
  using namespace sv;
  if (!k_cache || !v_cache || !block_table || !seq_lens || !start || !k_out || !v_out)
    return fail(SV_ERR_INVALID_ARG, "kv_block_gather_q4: null pointer argument");
  if (B < 0 || n_rows < 0 || H_kv < 1 || d_head < 1 || block_size < 1 || num_blocks < 1 || max_blocks_per_seq < 1)
    return fail(SV_ERR_INVALID_ARG, "kv_block_gather_q4: bad sizes");
  if (out_dtype != SV_F32 && out_dtype != SV_BF16)
    return fail(SV_ERR_UNSUPPORTED, "kv_block_gather_q4: rows are read back as f32 or bf16");
  if (B > 65535 || H_kv > 65535) return fail(SV_ERR_UNSUPPORTED, "kv_block_gather_q4: B or H_kv too large");
  if (!capacity_ok(max_blocks_per_seq, block_size))
    return fail(SV_ERR_UNSUPPORTED, "kv_block_gather_q4: max_blocks_per_seq * block_size must be below 2^30");
  Q4GatherArgs a = {};
  const sv_status rc = q4_check("kv_block_gather_q4", k_cache, v_cache, layout, H_kv, d_head, block_size,
                                &a.block_stride, &a.head_stride);
  if (rc != SV_OK) return rc;
  if (B == 0 || n_rows == 0) return ok();
  a.cache[0] = static_cast<const uint8_t *>(k_cache); a.cache[1] = static_cast<const uint8_t *>(v_cache);
  a.out[0] = k_out; a.out[1] = v_out; a.block_table = block_table; a.seq_lens = seq_lens; a.start = start;
  a.max_blocks = max_blocks_per_seq; a.n_rows = n_rows; a.H_kv = H_kv; a.bs = block_size;
  a.num_blocks = num_blocks; a.status = dev_status;
  a.pages = (int)(((int64_t)n_rows + block_size - 2) / block_size + 1);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (out_dtype == SV_F32) return launch_gather_q4_d<float>(a, d_head, B, s);
  return launch_gather_q4_d<__nv_bfloat16>(a, d_head, B, s);
}
