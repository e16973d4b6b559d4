// Verify attention with the keys on the lanes, what its kernels over a 4-bit and
// over an 8-bit block-scaled cache share: d_head 128, 16-token blocks, bf16
// queries. S^T = K Q^T has a key per lane of tensor memory, O^T = V^T P'^T a head
// dim, and the query rows of a kv head are the columns of both.
//
// Work: the tiles of all sequences end to end are cut into equal ranges, one
// per SM and kv head (and row group); each CTA streams through the sequences of
// its range, and a range that ends inside a sequence leaves fp32 partials for
// the merge. Included by one source file per kernel: the kernels here are
// internal to each.
#pragma once

#include <algorithm>
#include <mutex>

#include "q4.cuh"
#include "tc5.cuh"

namespace sv {
namespace {

constexpr int kD = 128;                    // head dim
constexpr int kBS = 16;                    // block size
constexpr int kTP = 8;                     // blocks per tile
constexpr int kTK = kTP * kBS;             // keys per tile
constexpr int kChunk = 8, kChunks = 4;     // tiles of a chunk of block offsets, and chunks in shared memory
constexpr int kFirst = 1, kLast = 2, kEnd = 4, kSecond = 8;   // of a tile: the sequence's first or last here, its step's last or second
constexpr int kWhole = 1, kOpening = 2;     // of an item: the whole sequence, the first of its CTA
constexpr float kUnset = 1e30f;            // minus the reference of a row that has met no key

// Query rows of a CTA that the first softmax warpgroup takes: up to 8 it takes
// all, so that a step's fixed work is done once (64 sequences of 1024-8192 keys,
// captured: 4 rows 90.3 against 97.4 us, 8 rows 96.4 against 97.4; up to 16 it
// would be 106.7 against 104.6 with 16 rows, 105.6 against 104.6 with 12).
constexpr int kAlone = 8;
// (of W warpgroups; row w * kl_first + c is row c of warpgroup w)
__host__ __device__ inline int kl_first(int rows, int W = 2) { return rows <= kAlone ? rows : (rows + W - 1) / W; }

struct KlParams {
  const void *q;
  void *out;
  const uint8_t *k_cache, *v_cache;
  const int32_t *block_table, *seq_lens;
  float *ws_acc;      // [2 CTAs][Rg][kD] partials (entry 2c: CTA c's first sequence, 2c + 1: its last)
  float *ws_ml;       // [2 CTAs][Rg][2]
  int4 *ws_split;     // per range: the sequence whose first cut is the range's start (b, first tile, tiles, T), or b = -1
  uint8_t *ws_q;      // per (sequence, kv head and row group): its Q as the kernel's shared memory holds it
  float *ws_qs;       // [2 kN + 4] per entry: the rows' sums, the power of two that undoes the scaling (or -1: every row
                      // has its own), and from kN + 4 on the rows' own
  int32_t *status;
  int64_t block_stride, head_stride;
  int B, n_new, H_q, H_kv, G, R;
  int Rg, RG;         // query rows of a CTA, and row groups per kv head
  int NR;             // ranges
  int max_blocks, num_blocks, window, sinks;
  float scale_log2;   // softmax_scale * log2(e)
  uint64_t wait_ns;
  unsigned withhold;
};

template <int NC, int W = 2> struct KlCfg {   // NC query rows per softmax warpgroup, W of these
  static constexpr int kCols = (NC + 7) / 8 * 8, kN = (W * kCols + 15) / 16 * 16;   // columns of S and O
  static constexpr int kT = W * NC > 48 ? 1 : 2;   // tiles of a softmax step (their scores stay in registers)
  static constexpr int kQ = kN * 256;   // the two e4m3 terms of a row, 128 bytes each
};

// A sequence's part of a CTA's range.
struct KlItem {
  int b, L, tile0, ntiles;
  KeySpan span;
  bool whole;      // the whole sequence: written directly
  bool first;      // the CTA's first item
};
// Walks the range; the next sequence's length is loaded one item ahead.
struct KlWalk {
  int b, off, left, L;
  bool first;
};

__device__ __forceinline__ int kl_tiles(const KlParams &P, int L) {
  if (L < P.n_new || L > P.max_blocks * kBS) return 0;
  return (key_span(L, P.n_new, P.window, P.sinks, kBS).nblk + kTP - 1) / kTP;
}

__device__ __forceinline__ KlWalk kl_walk(const KlParams &P, const int4 &w) {
  KlWalk k = {w.x, w.y, w.z, 0, true};
  if (k.left > 0 && k.b < P.B) k.L = P.seq_lens[k.b];
  return k;
}

__device__ __forceinline__ bool kl_next(const KlParams &P, KlWalk &w, KlItem &it) {
  if (w.left <= 0) return false;
  int nt;
  for (;;) {   // sequences with invalid lengths hold no tiles
    if (w.b >= P.B) return false;
    nt = kl_tiles(P, w.L);
    if (nt > 0) break;
    ++w.b;
    w.L = w.b < P.B ? P.seq_lens[w.b] : 0;
  }
  const int take = min(nt - w.off, w.left);
  it.b = w.b;
  it.L = w.L;
  it.tile0 = w.off;
  it.ntiles = take;
  it.span = key_span(w.L, P.n_new, P.window, P.sinks, kBS);
  it.whole = w.off == 0 && take == nt;
  it.first = w.first;
  w.first = false;
  w.left -= take;
  w.off = 0;
  ++w.b;
  w.L = w.left > 0 && w.b < P.B ? P.seq_lens[w.b] : 0;
  return true;
}

// One warp: range r of the tile sequence as (b, first tile within b, tiles),
// and the split record of the range's start; T is the number of tiles.
__device__ int4 kl_range(const KlParams &P, int r, int64_t T, int4 &split) {
  const int lane = threadIdx.x & 31;
  const int64_t t0 = r * T / P.NR, t1 = (r + 1) * T / P.NR;
  int4 w = make_int4(0, 0, 0, 0);
  split = make_int4(-1, 0, 0, 0);
  if (t1 <= t0) return w;
  int64_t A = 0;
  for (int b0 = 0; b0 < P.B; b0 += 128) {   // four sequences a lane
    int nt[4], own = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int b = b0 + 4 * lane + k;
      nt[k] = b < P.B ? kl_tiles(P, P.seq_lens[b]) : 0;
      own += nt[k];
    }
    int incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, A + incl > t0);
    if (hit) {
      const int src = __ffs(hit) - 1;
      int off = (int)(t0 - (A + __shfl_sync(0xffffffffu, incl - own, src))), k = 0, n = nt[0];
#pragma unroll
      for (int e = 1; e < 4; ++e) {   // (lane src: the sequence among its four)
        if (k == e - 1 && off >= n) {
          off -= n;
          n = nt[e];
          k = e;
        }
      }
      off = __shfl_sync(0xffffffffu, off, src);
      n = __shfl_sync(0xffffffffu, n, src);
      const int b = b0 + 4 * src + __shfl_sync(0xffffffffu, k, src);
      w = make_int4(b, off, (int)(t1 - t0), 0);
      // a range that starts inside a sequence is its first cut if one range
      // holds all its tiles before (tile x lies in range ((x + 1) NR - 1) / T)
      const int64_t first = t0 - off;
      if (off > 0 && (t0 * P.NR - 1) / T == ((first + 1) * P.NR - 1) / T) split = make_int4(b, (int)first, n, (int)T);
      return w;
    }
    A += __shfl_sync(0xffffffffu, incl, 31);
  }
  return w;
}

// One warp: the tiles of all sequences, and whether a length is out of range.
__device__ int64_t kl_all_tiles(const KlParams &P, bool &bad) {
  const int lane = threadIdx.x & 31;
  int own = 0;   // (all tiles together are below 2^30)
  bad = false;
#pragma unroll 4
  for (int b = lane; b < P.B; b += 32) {
    const int L = P.seq_lens[b];
    own += kl_tiles(P, L);
    bad = bad || L < P.n_new || L > P.max_blocks * kBS;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) own += __shfl_xor_sync(0xffffffffu, own, o);
  const int64_t T = own;
  return T;
}

// Before the attention: where the ranges cut sequences (the first CTAs, a warp a range), and the query
// rows of every (sequence, kv head and row group) as two e4m3 terms in the
// layout of the K-major 128-byte-swizzled operand, scaled by one power of two
// that brings the largest finite element of the entry to [2^7, 2^8). Where a
// row's own largest element lies more than 2^kNear below that (rows of padding may
// hold anything), every row has a power of its own, so that each keeps 2^-10 of its
// largest element whatever lies beside it. The kernel then takes a sequence's Q
// with one bulk copy: converted there, by one warp, it took 20,000 cycles a
// sequence.
constexpr int kPrepWarps = 4;
constexpr int kNear = 6;
// NIB (4-bit codes): the dims in the order in which codes are spread, with the
// rows' sums; otherwise in their own order. An infinite element would saturate to
// a finite term: it becomes NaN, so that its row's scores and output are NaN (with
// NIB the row's sum carries it).
template <int NC, int W, bool NIB>
__global__ void __launch_bounds__(32 * kPrepWarps) kl_prep_kernel(const __grid_constant__ KlParams P) {
  using Cfg = KlCfg<NC, W>;
  constexpr int N = Cfg::kN, CP = Cfg::kCols;
  constexpr int kPass = N / (2 * kPrepWarps);   // half a warp a row and pass
  __shared__ uint32_t s_top[kPrepWarps], s_low[kPrepWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nrange = (P.NR + kPrepWarps - 1) / kPrepWarps;
  pdl_trigger();
  if ((int)blockIdx.x < nrange) {
    // (the lengths are the caller's: read before the wait on the previous kernel)
    bool bad;
    const int64_t T = kl_all_tiles(P, bad);
    const int r = blockIdx.x * kPrepWarps + warp;
    int4 split = make_int4(-1, 0, 0, 0);
    if (r < P.NR) kl_range(P, r, T, split);
    pdl_wait();   // the previous kernel may still read this workspace
    if (blockIdx.x == 0 && warp == 0 && bad) atomic_or_status(P.status, SV_DEV_BAD_SEQ_LEN);
    if (r < P.NR && lane == 0) P.ws_split[r] = split;
    return;
  }
  pdl_wait();
  const int64_t ent = (int64_t)blockIdx.x - nrange;
  const int Hp = P.H_kv * P.RG;
  const int gp = (int)(ent % Hp), b = (int)(ent / Hp);
  const int g = gp / P.RG, row0 = (gp % P.RG) * P.Rg;
  const int rows = min(P.Rg, P.R - row0), live0 = kl_first(rows, W);
  const int c8 = lane & 15;
  uint4 v[kPass];
  // largest finite elements (their bits): of each row, of the entry, and of its smallest row but those of zeros
  uint32_t rtop[kPass], top = 0, low = 0x7f800000u;
#pragma unroll
  for (int k = 0; k < kPass; ++k) {
    const int col = (k * kPrepWarps + warp) * 2 + (lane >> 4);
    const int w = col / CP, c = col - w * CP;
    v[k] = make_uint4(0u, 0u, 0u, 0u);
    if (c < min(rows - w * live0, live0)) {
      const int r = row0 + w * live0 + c, j = r / P.G;
      const int64_t at = ((int64_t)b * P.n_new + j) * P.H_q + g * P.G + (r - j * P.G);
      v[k] = static_cast<const uint4 *>(P.q)[at * 16 + c8];
    }
  }
#pragma unroll
  for (int k = 0; k < kPass; ++k) {
    const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
    rtop[k] = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t lo = (w[e] << 16) & 0x7fffffffu, hi = w[e] & 0x7fff0000u;
      if (lo < 0x7f800000u) rtop[k] = max(rtop[k], lo);
      if (hi < 0x7f800000u) rtop[k] = max(rtop[k], hi);
    }
  }
#pragma unroll
  for (int o = 8; o > 0; o >>= 1)   // (half a warp a row)
#pragma unroll
    for (int k = 0; k < kPass; ++k) rtop[k] = max(rtop[k], __shfl_xor_sync(0xffffffffu, rtop[k], o));
#pragma unroll
  for (int k = 0; k < kPass; ++k) {
    top = max(top, rtop[k]);
    if (rtop[k] != 0) low = min(low, rtop[k]);
  }
  top = __reduce_max_sync(0xffffffffu, top);
  low = __reduce_min_sync(0xffffffffu, low);
  if (lane == 0) {
    s_top[warp] = top;
    s_low[warp] = low;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kPrepWarps; ++k) {
    top = max(top, s_top[k]);
    low = min(low, s_low[k]);
  }
  const bool own = (int)(top >> 23) - (int)(low >> 23) > kNear;
  auto power = [](uint32_t t) { return min(117, max(-113, (int)(t >> 23) - 127)); };   // (all powers stay normal)
  // 2^(7 - power) of Q, and 2^-9 of 4-bit codes
  auto undo = [](int ex) { return __uint_as_float((uint32_t)(127 - 7 + (NIB ? 9 : 0) + ex) << 23); };
  uint8_t *img = P.ws_q + ent * Cfg::kQ;
  float *qs = P.ws_qs + ent * (2 * N + 4);
#pragma unroll
  for (int k = 0; k < kPass; ++k) {
    const int col = (k * kPrepWarps + warp) * 2 + (lane >> 4);
    const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
    float x[8], sum = 0.f;
    const int ex = power(own ? rtop[k] : top);
    const float up = __uint_as_float((uint32_t)(127 + 7 - ex) << 23);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = __uint_as_float(w[e] << 16);
      x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) sum += x[e];
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    uint32_t hi[2], lo[2];   // dims 0 2 4 6, then 1 3 5 7 in the order of 4-bit codes; else 0 1 2 3, then 4 5 6 7
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      hi[e] = lo[e] = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float y0 = x[NIB ? 4 * h + e : 4 * e + 2 * h] * up, y1 = x[NIB ? 4 * h + 2 + e : 4 * e + 2 * h + 1] * up;
        if constexpr (!NIB) {   // (what is finite is below 2^8)
          y0 += y0 - y0;
          y1 += y1 - y1;
        }
        const uint32_t c = f32x2_to_e4m3x2(y0, y1);
        const uint32_t f = e4m3x2_to_f16x2((uint16_t)c);
        const float2 hv = __half22float2(*reinterpret_cast<const __half2 *>(&f));
        hi[e] |= c << (16 * h);
        lo[e] |= f32x2_to_e4m3x2(y0 - hv.x, y1 - hv.y) << (16 * h);
      }
    }
    uint8_t *dst = img + col * 128 + (((c8 >> 1) ^ (col & 7)) << 4) + (c8 & 1) * 8;
    *reinterpret_cast<uint2 *>(dst) = make_uint2(hi[0], hi[1]);
    *reinterpret_cast<uint2 *>(dst + N * 128) = make_uint2(lo[0], lo[1]);
    if (c8 == 0) {
      qs[col] = sum;
      if (own) qs[N + 4 + col] = undo(ex);
    }
  }
  if (threadIdx.x == 0) qs[N] = own ? -1.f : undo(power(top));
}

__device__ __forceinline__ bool bar_or(int id, int threads, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)v), "r"(id), "r"(threads)
      : "memory");
  return r != 0;
}

// Bounded wait; gives up at once after any earlier one of the CTA gave up. (Naps
// of 20 to 800 ns between the tries change neither the time nor the number of
// instructions: try_wait itself sleeps.)
__device__ __forceinline__ bool kl_wait(uint64_t *bar, uint32_t phase, volatile int *abort_flag, uint64_t limit_ns) {
  if (mbar_try_wait(bar, phase)) return true;
  const uint64_t t0 = global_ns();
  do {
    if (mbar_try_wait(bar, phase)) return true;
  } while (!*abort_flag && global_ns() - t0 <= limit_ns);
  *abort_flag = 1;
  return false;
}

// Both at once: the first tries overlap.
__device__ __forceinline__ bool kl_wait2(uint64_t *a, uint32_t phase_a, uint64_t *b, uint32_t phase_b, volatile int *abort_flag,
                                         uint64_t limit_ns) {
  const bool da = mbar_try_wait(a, phase_a), db = mbar_try_wait(b, phase_b);
  if (da && db) return true;
  return (da || kl_wait(a, phase_a, abort_flag, limit_ns)) && (db || kl_wait(b, phase_b, abort_flag, limit_ns));
}

// true in one lane of a converged warp, in a form that keeps the code around it
// uniform for the compiler
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ float lg2f(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcpf(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// kind::f8f6f4 (e4m3 A and B, 32 elements of K per MMA), A from tensor memory
__device__ __forceinline__ void t5_mma_ts_f8(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
               "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
               "r"(a), "l"(b), "r"(idesc), "r"(acc));
}

// Sums, or maxima (NaN left out), of v[0..NV) over the warp's lanes. While their
// number is even, each step exchanges the half of the values that the other lane
// keeps; lane l is left with those of n values from `at` on.
template <int NV, bool MAX, int O = 16>
__device__ __forceinline__ void warp_joined(float *v, int lane, int &at, int &n) {
  auto join = [](float a, float b) { return MAX ? fmaxf(a, b) : a + b; };
  if constexpr (O == 0) {
    n = NV;
  } else if constexpr (NV % 2 == 0) {
    constexpr int H = NV / 2;
    const bool up = lane & O;
#pragma unroll
    for (int k = 0; k < H; ++k) {
      const float send = up ? v[k] : v[k + H], keep = up ? v[k + H] : v[k];
      v[k] = join(keep, __shfl_xor_sync(0xffffffffu, send, O));
    }
    if (up) at += H;
    warp_joined<H, MAX, O / 2>(v, lane, at, n);
  } else {
#pragma unroll
    for (int k = 0; k < NV; ++k) v[k] = join(v[k], __shfl_xor_sync(0xffffffffu, v[k], O));
    warp_joined<NV, MAX, O / 2>(v, lane, at, n);
  }
}
template <int NV>
__device__ __forceinline__ void warp_sums(float *v, int lane, int &at, int &n) { warp_joined<NV, false>(v, lane, at, n); }

// Largest of the warp's values (NaN left out)
__device__ __forceinline__ float warp_top(float x) {
  float m;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x));
  return m;
}

// N columns of this warp's lanes, N a multiple of 4
__device__ __forceinline__ void t5_ld8(uint32_t taddr, uint32_t *r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void t5_ld4(uint32_t taddr, uint32_t *r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(taddr));
}
template <int N>
__device__ __forceinline__ void t5_ldn(uint32_t taddr, uint32_t (&r)[N]) {
  constexpr int a = N / 16 * 16, b = a + (N - a) / 8 * 8;
#pragma unroll
  for (int k = 0; k < a; k += 16) t5_ld16(taddr + k, *reinterpret_cast<uint32_t(*)[16]>(r + k));
  if constexpr (b > a) t5_ld8(taddr + a, r + a);
  if constexpr (N > b) t5_ld4(taddr + b, r + b);
}
// Keeps the compiler from using loaded columns ahead of the wait before this.
template <int N>
__device__ __forceinline__ void keep_after(float (&r)[N]) {
#pragma unroll
  for (int k = 0; k < N; k += 4) asm volatile("" : "+f"(r[k]), "+f"(r[k + 1]), "+f"(r[k + 2]), "+f"(r[k + 3]));
}
__device__ __forceinline__ void t5_st4(uint32_t taddr, const uint32_t *r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3])
               : "memory");
}
__device__ __forceinline__ void t5_st8(uint32_t taddr, const uint32_t *r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

template <int N>
__device__ __forceinline__ void t5_stn(uint32_t taddr, const uint32_t (&r)[N]) {
  constexpr int a = N / 16 * 16, b = a + (N - a) / 8 * 8;
#pragma unroll
  for (int k = 0; k < a; k += 16) t5_st16(taddr + k, *reinterpret_cast<const uint32_t(*)[16]>(r + k));
  if constexpr (b > a) t5_st8(taddr + a, r + a);
  if constexpr (N > b) t5_st4(taddr + b, r + b);
}

// Columns of S times their rows' powers of two, where they lie (nt tiles)
template <int NC, int N>
__device__ __noinline__ void kl_scale_rows(uint32_t s_col, int nt, const float *qf) {
  t5_fence_after();
#pragma unroll 1
  for (int h = 0; h < nt; ++h)
#pragma unroll 1
    for (int c = 0; c < NC; c += 4) {
      const float4 f = *reinterpret_cast<const float4 *>(qf + c);
      float x[4];
      t5_ld4(s_col + h * N + c, reinterpret_cast<uint32_t *>(x));
      t5_wait_ld();
      keep_after<4>(x);
      x[0] *= f.x; x[1] *= f.y; x[2] *= f.z; x[3] *= f.w;
      t5_st4(s_col + h * N + c, reinterpret_cast<const uint32_t *>(x));
    }
  t5_wait_st();
}

// Merge of the sequences that more than one range holds: CTA (range r, kv head
// and row group, eight rows) leaves at once unless r's start is the first cut
// of a sequence. Its pieces come from ranges r - 1 (the last item of its CTA,
// or the first if that range starts with the sequence), r, r + 1, ... (first
// items); a warp takes a row, lane l the head dims 4l .. 4l + 3, and loads
// eight pieces at once.
constexpr int kMergeWarps = 8;
__global__ void __launch_bounds__(32 * kMergeWarps) kl_merge_kernel(const __grid_constant__ KlParams P) {
  pdl_wait();
  pdl_trigger();
  const int Hp = P.H_kv * P.RG;
  const int r = 1 + blockIdx.x / Hp, gp = blockIdx.x % Hp;
  const int4 sp = P.ws_split[r];
  if (sp.x < 0) return;
  const int lane = threadIdx.x & 31;
  const int g = gp / P.RG, row0 = (gp % P.RG) * P.Rg;
  const int row = blockIdx.y * kMergeWarps + (threadIdx.x >> 5);
  if (row >= min(P.Rg, P.R - row0)) return;
  const int64_t T = sp.w, A = sp.y, end = A + sp.z;
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kMB = 8;
  const int last = (int)((end * P.NR - 1) / T);   // the range that holds the last tile
  // empty ranges before r hold nothing: the piece before the cut is that of the range with tile A
  const int first = (int)(((A + 1) * P.NR - 1) / T);
  for (int e0 = first; e0 <= last; e0 += kMB) {
    float me[kMB], le[kMB];
    float4 va[kMB];
#pragma unroll
    for (int k = 0; k < kMB; ++k) {
      const int e = e0 + k;
      const int64_t t0 = (int64_t)e * T / P.NR, t1 = (int64_t)(e + 1) * T / P.NR;
      me[k] = -INFINITY;
      le[k] = 0.f;
      va[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (e <= last && t1 > t0) {
        const int64_t at = (2 * ((int64_t)e * Hp + gp) + (t0 < A ? 1 : 0)) * P.Rg + row;
        me[k] = P.ws_ml[2 * at];
        le[k] = P.ws_ml[2 * at + 1];
        va[k] = reinterpret_cast<const float4 *>(P.ws_acc + at * kD)[lane];
      }
    }
    float mn = m;
#pragma unroll
    for (int k = 0; k < kMB; ++k) mn = fmaxf(mn, me[k]);
    const float base = mn == -INFINITY ? 0.f : mn;
    const float a = ex2f(m - base);
    l *= a;
    acc.x *= a; acc.y *= a; acc.z *= a; acc.w *= a;
#pragma unroll
    for (int k = 0; k < kMB; ++k) {
      const float x = ex2f(me[k] - base);
      l = fmaf(le[k], x, l);
      acc.x = fmaf(va[k].x, x, acc.x);
      acc.y = fmaf(va[k].y, x, acc.y);
      acc.z = fmaf(va[k].z, x, acc.z);
      acc.w = fmaf(va[k].w, x, acc.w);
    }
    m = mn;
  }
  const float inv = 1.f / l;
  const int rr = row0 + row, j = rr / P.G;
  const int64_t o = ((int64_t)sp.x * P.n_new + j) * P.H_q + g * P.G + (rr - j * P.G);
  uint2 w;
  w.x = pack2<false>(acc.x * inv, acc.y * inv);
  w.y = pack2<false>(acc.z * inv, acc.w * inv);
  reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(P.out) + o * kD)[lane] = w;
}

inline int kl_sms() {
  static int n = 0;
  static std::once_flag once;
  std::call_once(once, [] {
    int dev = 0;
    cudaGetDevice(&dev);
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) n = 148;
  });
  return n;
}

struct KlPlan {
  bool tc;
  int R, RG, Rg, NR, C;
};

inline KlPlan kl_plan(int B, int n_new, int H_q, int H_kv, int d, int max_blocks, int bs, sv_dtype qd, int window, int sinks,
               int64_t max_rows) {
  KlPlan p = {};
  const int span = span_blocks_max(max_blocks, n_new, window, sinks, bs);
  const int64_t tiles = (int64_t)std::max(B, 1) * ((span + kTP - 1) / kTP);
  const int64_t R = (int64_t)n_new * (H_q / H_kv);
  p.tc = qd == SV_BF16 && d == kD && bs == kBS && R <= max_rows && tiles < (1ll << 30) &&
         (int64_t)B * n_new * H_q < (1ll << 30);
  if (!p.tc) return p;
  p.R = (int)R;
  p.RG = (p.R + 63) / 64;                // at most 64 query rows a CTA (the registers of the softmax warps)
  p.Rg = (p.R + p.RG - 1) / p.RG;
  const int64_t Hp = (int64_t)H_kv * p.RG;
  // Four tiles in all stay in one range, which needs no merge (captured, with the
  // replay's own 5 us: 256 keys, one position, 13.4 against 17.5 us with 8 kv
  // heads and 14.4 against 16.6 with 40; 512 keys 15.5 against 16.5 and 15.5
  // against 18.6; 8 positions of 64/8 heads 19.6 against 23.7 at 256 keys and
  // 22.6 against 24.7 at 512. Up to eight tiles 1000 keys gain nothing.) A range
  // per SM and kv head leaves SMs idle where the heads do not divide them: 40
  // heads take 120 of 152, 77 and more have one range each (80 heads as long as
  // 152: 294 and 298 us for 16 sequences of 4000).
  p.NR = tiles <= 4 ? 1 : (int)std::max<int64_t>(1, std::min<int64_t>(kl_sms() / Hp, tiles));
  p.C = (int)(p.NR * Hp);
  return p;
}

// Columns of S and O: a softmax warpgroup's rows in steps of 8, all together in steps of 16
inline int kl_cols(const KlPlan &p, int W = 2) { return (W * ((kl_first(p.Rg, W) + 7) / 8 * 8) + 15) / 16 * 16; }

inline size_t kl_ws_bytes(const KlPlan &p, int B, int H_kv, int W = 2) {
  const size_t ent = (size_t)2 * p.C * p.Rg, qent = (size_t)B * H_kv * p.RG, n = kl_cols(p, W);
  return align_up(ent * kD * sizeof(float), 256) + align_up(ent * 2 * sizeof(float), 256) +
         align_up((size_t)p.NR * sizeof(int4), 256) + align_up(qent * n * 256, 256) +
         align_up(qent * (2 * n + 4) * sizeof(float), 256);
}

}  // namespace
}  // namespace sv
