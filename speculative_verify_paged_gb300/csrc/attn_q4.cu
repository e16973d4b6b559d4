// spec_verify_attn_q4 on the tensor cores: paged GQA verify attention over a
// 4-bit cache (record layout: q4.cuh), d_head 128, 16-token blocks, bf16
// queries.
//
// Mathematics. With K_t = s_t c_t + m_t and V_t = s'_t c'_t + m'_t (c, c' codes
// in 0..15, one scale and minimum per key), for query row r
//   x_rt = scale (s_t (q_r . c_t) + m_t sum(q_r)),
//   p'_rt = s'_t 2^(x_rt - ref_r)            (log2 domain, ref_r a running reference)
//   out_r = [sum_t p'_rt (c'_t - z_t) + sum_t p'_rt (m'_t / s'_t + z_t)] / sum_t p'_rt / s'_t
// so both products run on the bare codes and the scales enter per key. z_t is 0
// for even keys and 15 for odd ones, whose terms are taken as -p' (15 - c'). (The
// tensor cores' accumulation rounds towards zero: with terms of one sign the
// first sum grows to some 8 sum p', and at 128K keys, where the outputs are
// averages near zero, its rounding errors reached 1 % of the outputs.)
//
// Codes as operands. A K code in the low four bits of a byte is, read as e4m3,
// the code times 2^-9 exactly (0 to 7 are subnormals, 8 to 15 the first normal
// binade), so a word of eight codes becomes two words of e4m3 with three
// instructions: Q K^T runs in kind::f8f6f4 with each query row as two e4m3 terms
// (hi + lo: 8 bits down to 2^-9 of the largest element scaled with it, an error
// of 2^-17 of that one below). V codes are subnormals of f16 in bits 0-3 of a
// half, or 4-7: then 16 times as large, and those keys have weights 16 times
// smaller; a word becomes four with five instructions (15 - c' is the
// complement). P V runs in kind::f16. Both spread the codes of a word over several registers, so the
// other operand of each product is stored in that order.
// Keys on the lanes. The M = 128 side of both products is the cache: S^T = C Q^T
// has a key per lane, O^T = C'^T P'^T a head dim per lane, and N is the number
// of query rows in steps of 16 (up to 64), so little tensor-core work is padding
// whatever the GQA group. The A operand is written by the thread that owns its lane, from
// its own 64 bytes of codes, straight into tensor memory; shared memory holds
// only the raw records, Q and P'. A K record is slot-major and a V record
// dim-major for this reason.
//
// What bounds it: 136 bytes per key and kv head leave about 820 SM cycles per
// 128-key tile at the measured HBM bandwidth, for 2 x 128 x 128 codes to unpack
// and 128 R exponentials. Measured: 64 sequences of 1024-8192 keys, 5 positions,
// 64/8 heads take 126.4 us (330 MB, 2.6 TB/s; 49 us at the bandwidth), 128K keys
// with 8 positions 81.5 us, about 1700 cycles a tile of 40 rows. A tile takes 4150
// warp instructions (V 485, K 361, the exponentials and P' 625, the scores 700,
// the rest copies, waits and bookkeeping) at 60 % of the issue slots; the softmax
// warps are the ones the others wait for, and each part that is taken out for a
// test gains 3 to 9 %.
//
// Work: the tiles of all sequences end to end are cut into equal ranges, one
// per SM and kv head; each CTA (one per SM) streams through the sequences of its
// range without draining the pipeline. A range that ends inside a sequence
// leaves fp32 partials for the merge.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>
#include <mutex>
#include <type_traits>

#include "q4.cuh"
#include "tc5.cuh"

namespace sv {
namespace {

constexpr int kD = 128;                    // head dim
constexpr int kBS = 16;                    // block size
constexpr int kTP = 8;                     // blocks per tile
constexpr int kTK = kTP * kBS;             // keys per tile
constexpr int kCodes = kBS * kD / 2;       // code bytes of a record
constexpr int kNS = 3;                     // stages of a K or V warp's ring of codes (2 KB each)
// The keys' scales, unpacked: a K warp writes those of tile u before it hands
// over the codes, after Q K^T of tile u - 2; that waited for the softmax of the
// step before the last, so every tile up to u - 6 has been read.
constexpr int kScales = 8;
constexpr int kScaleBytes = kTK * 20;      // a float4 and a float a key
constexpr int kChunk = 8, kChunks = 4;     // tiles of a chunk of block offsets, and chunks in shared memory
constexpr int kPBytes = kTK * 128;         // a P' buffer: 128 bytes (64 columns of f16) a key
constexpr int kWarps = 28;
constexpr int kKWarp = 8, kVWarp = 16, kPageWarp = 24, kQkWarp = 25, kPvWarp = 26, kQWarp = 27;
constexpr int kRegs = 72;                  // a thread at the launch
constexpr int kFirst = 1, kLast = 2, kEnd = 4, kSecond = 8;   // of a tile: the sequence's first or last here, its step's last or second
constexpr int kWhole = 1, kOpening = 2;     // of an item: the whole sequence, the first of its CTA
constexpr float kUnset = 1e30f;            // minus the reference of a row that has met no key
// P' is f16. A row's reference puts its largest weight at 2^kTop and moves once
// one exceeds 2^kMove (f16 ends at 65504), so weights keep f16's 11 bits down to
// 2^-21 of the largest (odd keys, stored 16 times smaller: 2^-17) and an absolute
// error of 2^-32 (2^-28) of it below. A key whose weight f16 loses counts as an
// end of its row's range 15 s', since the sums below take the fp32 weight: n such
// keys move an output by at most n 2^-28 of that range. With the largest weight at
// 1 and 128K keys beside one that holds 97 % of the weight, that was 4 % of the
// output; it is 4e-6 now.
constexpr float kTop = 7.f, kMove = 15.f;

// Query rows of a CTA that the first softmax warpgroup takes: up to 8 it takes
// all, so that a step's fixed work is done once (64 sequences of 1024-8192 keys,
// captured: 4 rows 90.3 against 97.4 us, 8 rows 96.4 against 97.4; up to 16 it
// would be 106.7 against 104.6 with 16 rows, 105.6 against 104.6 with 12).
constexpr int kAlone = 8;
__host__ __device__ inline int q4_first(int rows) { return rows <= kAlone ? rows : (rows + 1) / 2; }

struct Q4Params {
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

template <int NC> struct Q4Cfg {   // NC query rows per softmax warpgroup
  static constexpr int kCols = (NC + 7) / 8 * 8, kN = 2 * kCols;   // columns of S and O
  static constexpr int kT = NC > 24 ? 1 : 2;   // tiles of a softmax step (their scores stay in registers)
  // Registers: the K, V and service warps hand over theirs so that the softmax
  // warps hold a step's scores and two sums per column. 144 / 40 against 168 / 32
  // (64 sequences of 1024-8192 keys, captured, resolution 1 us): 89.2 and 91.2 us
  // with 4 columns, 104.6 and 105.6 with 8, 113.8 and 115.8 with 12, 122.0 and
  // 125.0 with 16, 136.3 both with 20, 152.7 and 148.6 with 24, 197.8 and 186.5
  // with 32 (spills on one side or the other).
  static constexpr int kRegsSoftmax = NC <= 20 ? 144 : 168, kRegsOther = NC <= 20 ? 40 : 32;
  static_assert(256 * kRegsSoftmax + 32 * (kWarps - 8) * kRegsOther <= 32 * kWarps * kRegs, "registers");
  static constexpr int kQ = kN * 256;   // the two e4m3 terms of a row, 128 bytes each
  static constexpr uint32_t kKCol = 0, kVCol = 64, kSCol = 192, kOCol = 192 + 2 * kT * kN;   // (two O buffers)
  static constexpr int kSmem = 1024 + 2 * kQ + 2 * kT * kPBytes + 16 * kNS * 2048 + 8 * kNS * 256 + kScales * kScaleBytes;
  static_assert(kOCol + 2 * kN <= 512, "TMEM columns");
  static_assert(kSmem + 8192 <= 227 * 1024, "shared memory");
};

// A sequence's part of a CTA's range.
struct Q4Item {
  int b, L, tile0, ntiles;
  KeySpan span;
  bool whole;      // the whole sequence: written directly
  bool first;      // the CTA's first item
};
// Walks the range; the next sequence's length is loaded one item ahead.
struct Q4Walk {
  int b, off, left, L;
  bool first;
};

__device__ __forceinline__ int q4_tiles(const Q4Params &P, int L) {
  if (L < P.n_new || L > P.max_blocks * kBS) return 0;
  return (key_span(L, P.n_new, P.window, P.sinks, kBS).nblk + kTP - 1) / kTP;
}

__device__ __forceinline__ Q4Walk q4_walk(const Q4Params &P, const int4 &w) {
  Q4Walk k = {w.x, w.y, w.z, 0, true};
  if (k.left > 0 && k.b < P.B) k.L = P.seq_lens[k.b];
  return k;
}

__device__ __forceinline__ bool q4_next(const Q4Params &P, Q4Walk &w, Q4Item &it) {
  if (w.left <= 0) return false;
  int nt;
  for (;;) {   // sequences with invalid lengths hold no tiles
    if (w.b >= P.B) return false;
    nt = q4_tiles(P, w.L);
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
__device__ int4 q4_range(const Q4Params &P, int r, int64_t T, int4 &split) {
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
      nt[k] = b < P.B ? q4_tiles(P, P.seq_lens[b]) : 0;
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
__device__ int64_t q4_all_tiles(const Q4Params &P, bool &bad) {
  const int lane = threadIdx.x & 31;
  int own = 0;   // (all tiles together are below 2^30)
  bad = false;
#pragma unroll 4
  for (int b = lane; b < P.B; b += 32) {
    const int L = P.seq_lens[b];
    own += q4_tiles(P, L);
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
template <int NC>
__global__ void __launch_bounds__(32 * kPrepWarps) attn_q4_prep_kernel(const __grid_constant__ Q4Params P) {
  using Cfg = Q4Cfg<NC>;
  constexpr int N = Cfg::kN, CP = Cfg::kCols;
  constexpr int kPass = N / (2 * kPrepWarps);   // half a warp a row and pass
  __shared__ uint32_t s_top[kPrepWarps], s_low[kPrepWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nrange = (P.NR + kPrepWarps - 1) / kPrepWarps;
  pdl_trigger();
  if ((int)blockIdx.x < nrange) {
    // (the lengths are the caller's: read before the wait on the previous kernel)
    bool bad;
    const int64_t T = q4_all_tiles(P, bad);
    const int r = blockIdx.x * kPrepWarps + warp;
    int4 split = make_int4(-1, 0, 0, 0);
    if (r < P.NR) q4_range(P, r, T, split);
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
  const int rows = min(P.Rg, P.R - row0), live0 = q4_first(rows);
  const int c8 = lane & 15;
  uint4 v[kPass];
  // largest finite elements (their bits): of each row, of the entry, and of its smallest row but those of zeros
  uint32_t rtop[kPass], top = 0, low = 0x7f800000u;
#pragma unroll
  for (int k = 0; k < kPass; ++k) {
    const int col = (k * kPrepWarps + warp) * 2 + (lane >> 4);
    const int w = col / CP, c = col - w * CP;
    v[k] = make_uint4(0u, 0u, 0u, 0u);
    if (c < (w ? rows - live0 : live0)) {
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
  // 2^-9 of the codes and 2^(7 - power) of Q
  auto undo = [](int ex) { return __uint_as_float((uint32_t)(127 + 2 + ex) << 23); };
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
    uint32_t hi[2], lo[2];   // in the order of the codes: dims 0 2 4 6, then 1 3 5 7
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      hi[e] = lo[e] = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float y0 = x[4 * h + e] * up, y1 = x[4 * h + 2 + e] * up;
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
__device__ __forceinline__ bool q4_wait(uint64_t *bar, uint32_t phase, volatile int *abort_flag, uint64_t limit_ns) {
  if (mbar_try_wait(bar, phase)) return true;
  const uint64_t t0 = global_ns();
  do {
    if (mbar_try_wait(bar, phase)) return true;
  } while (!*abort_flag && global_ns() - t0 <= limit_ns);
  *abort_flag = 1;
  return false;
}

// true in one lane of a converged warp, in a form that keeps the code around it
// uniform for the compiler
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// 16-byte asynchronous copy
__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <int R> __device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R> __device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }

// eight K codes of a word -> two words of e4m3 (codes 0 2 4 6, then 1 3 5 7),
// each the code times 2^-9
__device__ __forceinline__ void spread_k(uint32_t w, uint32_t *o) {
  o[0] = w & 0x0F0F0F0Fu;
  o[1] = (w >> 4) & 0x0F0F0F0Fu;
}
// eight V codes of a word -> four f16 pairs (codes k and k + 4): a code times
// 2^-24 for even k, 15 minus the code times 2^-20 for odd k
__device__ __forceinline__ void spread_v(uint32_t w, uint32_t *o) {
  o[0] = w & 0x000F000Fu;
  o[1] = ~w & 0x00F000F0u;
  w >>= 8;
  o[2] = w & 0x000F000Fu;
  o[3] = ~w & 0x00F000F0u;
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

// Sums of v[0..NV) over the warp's lanes. While their number is even, each step
// exchanges the half of the values that the other lane keeps; lane l is left
// with the sums of n values from `at` on.
template <int NV, int O = 16>
__device__ __forceinline__ void warp_sums(float *v, int lane, int &at, int &n) {
  if constexpr (O == 0) {
    n = NV;
  } else if constexpr (NV % 2 == 0) {
    constexpr int H = NV / 2;
    const bool up = lane & O;
#pragma unroll
    for (int k = 0; k < H; ++k) {
      const float send = up ? v[k] : v[k + H], keep = up ? v[k + H] : v[k];
      v[k] = keep + __shfl_xor_sync(0xffffffffu, send, O);
    }
    if (up) at += H;
    warp_sums<H, O / 2>(v, lane, at, n);
  } else {
#pragma unroll
    for (int k = 0; k < NV; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], O);
    warp_sums<NV, O / 2>(v, lane, at, n);
  }
}

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

// Columns of S times their rows' powers of two, where they lie (nt tiles)
template <int NC, int N>
__device__ __noinline__ void q4_scale_rows(uint32_t s_col, int nt, const float *qf) {
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

// Warps 0-3 and 4-7: softmax (a key per thread and tile; each warpgroup half
// of the query rows, or the first all of them), later the epilogue (a head dim per thread). 8-15: K codes
// to tensor memory, 16-23: V codes (four warps per tile parity). 24: block
// offsets and flags of the tiles ahead. 25: issues Q K^T, owns the 512 TMEM
// columns (two K, two V, four S and two O buffers). 26: issues P V (one warp for
// both products took 1400 cycles a tile for its waits and commits alone). 27: Q
// of the next sequence.
// The softmax takes two tiles at a time (one with more than 48 rows, whose
// scores would not fit in registers): its waits, its vote and its fences cost as
// much as the arithmetic of a tile. (Four for up to 16 rows, with two or four V
// buffers, gained nothing.)
// Every warp copies what it reads: a K warp the two blocks that its keys lie
// in (and the keys' pairs of K and V, which it unpacks for the softmax), a V
// warp its 32 head dims of the tile's eight blocks; so a copy is waited for by
// its own warp alone. (Bulk copies of whole records were limited by their issue:
// 1088 bytes each, they reached 2.9 TB/s from one warp and 4.8 TB/s from sixteen.)
template <int NC>
__global__ void __launch_bounds__(32 * kWarps, 1) attn_q4_kernel(const __grid_constant__ Q4Params P) {
  using Cfg = Q4Cfg<NC>;
  constexpr int N = Cfg::kN, CP = Cfg::kCols, T = Cfg::kT;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t page_full[kChunks], page_empty[kChunks];
  // offsets of the blocks of the tiles ahead in 16-byte units, even blocks of a tile first
  __shared__ __align__(16) uint32_t s_off[kChunks * kChunk * kTP];
  __shared__ int s_flag[kChunks * kChunk];   // kFirst, kLast, kEnd, kSecond, blocks of the tile << 8
  __shared__ __align__(8) uint64_t kop_full[2], kop_empty[2], vop_full[2], vop_empty[2];
  __shared__ __align__(8) uint64_t s_full[2], p_full[2], pv_done[2], q_full[2], q_empty[2], o_free[2], drain[2];
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  __shared__ int4 s_work;
  // per row of the items in flight: sum(q), position (0 .. n_new - 1),
  // row of q and out, its own power of two; per item the power of two that undoes Q's scaling (-1: the rows have their own)
  __shared__ __align__(16) float s_qs[3][N], s_qf[3][N];
  __shared__ __align__(16) int s_pos[3][N];
  __shared__ int s_row[3][N];
  __shared__ float s_fold[3];
  __shared__ __align__(16) int4 s_item[3];   // first tile, tiles, length in span coordinates, kWhole | kOpening
  __shared__ __align__(16) float s_nb[N], s_a[N];   // minus the reference; the last factor of a rescale
  __shared__ float s_max[8][NC], s_red[8][2 * NC];
  __shared__ __align__(8) float2 s_fin[2][N];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int Hp = P.H_kv * P.RG;
  const int range = blockIdx.x / Hp, gp = blockIdx.x % Hp;
  const int g = gp / P.RG, row0 = (gp % P.RG) * P.Rg;
  const int rows = min(P.Rg, P.R - row0);       // live rows of this CTA
  const int live0 = q4_first(rows);             // of the first softmax warpgroup
  const int softmax_warps = live0 < rows ? 8 : 4;
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t q_smem = smem_u32(smem);
  const uint32_t p_smem = q_smem + 2 * Cfg::kQ;
  const uint32_t ring = p_smem + 2 * T * kPBytes;
  const uint32_t pairs = ring + 16 * kNS * 2048;      // the K warps' rings of (scale, minimum) pairs
  const uint32_t scales = pairs + 8 * kNS * 256;

  // Lengths and block numbers are the caller's: the ranges and the first block
  // offsets are worked out while the kernel before this one runs.
  if (warp == 0) {
    bool bad;
    int4 split;
    const int64_t all = q4_all_tiles(P, bad);
    const int4 w = q4_range(P, range, all, split);
    if (lane == 0) s_work = w;
  } else if (tid == 32) {
    for (int k = 0; k < kChunks; ++k) {
      mbar_init(&page_full[k], 1);
      mbar_init(&page_empty[k], 18);   // the K, V and MMA warps
    }
    for (int k = 0; k < 2; ++k) {
      mbar_init(&kop_full[k], 4);
      mbar_init(&kop_empty[k], 1);
      mbar_init(&vop_full[k], 4);
      mbar_init(&vop_empty[k], 1);
      mbar_init(&drain[k], 1);
      mbar_init(&q_full[k], 1);
      mbar_init(&q_empty[k], 1);
      mbar_init(&o_free[k], softmax_warps);
      // Q K^T of the step (its commit, and the issuing lane itself, which has seen
      // the K warps' scales), and P V of the step before the last
      mbar_init(&s_full[k], 3);
      mbar_init(&p_full[k], softmax_warps);
      mbar_init(&pv_done[k], 1);
    }
    abort_flag = 0;
    fence_mbarrier_init();
  } else if (warp == kQkWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base)),
                 "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  t5_fence_before();
  __syncthreads();
  t5_fence_after();
  const uint32_t tb = tmem_base;
  const int4 work = s_work;
  const int total = work.z;   // tiles of this CTA
  volatile int *abf = &abort_flag;
  // every stage, buffer and phase below follows the CTA's running tile count u

  // The blocks of tile u (u < total) for the copies of this warp, which takes
  // every step-th tile; done with a chunk's last tile it hands the chunk back.
  auto pages_of = [&](uint32_t u, uint32_t step, bool &ok) -> const uint32_t * {
    if (u % kChunk < step)
      ok = q4_wait(&page_full[u / kChunk % kChunks], (u / (kChunk * kChunks)) & 1, abf, P.wait_ns) && ok;
    return s_off + u % (kChunk * kChunks) * kTP;
  };
  auto pages_done = [&](uint32_t u, uint32_t step) {
    if (u % kChunk >= kChunk - step) {
      __syncwarp();
      if (lane == 0) mbar_arrive(&page_empty[u / kChunk % kChunks]);
    }
  };

  if (warp >= kPageWarp) regs_dec<Cfg::kRegsOther>();
  if (warp != kPageWarp) pdl_wait();
  pdl_trigger();
  if (warp == kPageWarp) {
    // ------------------------------------------------------- block numbers --
    Q4Walk wk = q4_walk(P, work);
    Q4Item it;
    bool have = q4_next(P, wk, it);
    int ti = 0;   // next tile of the item
    bool bad = false;
    const uint32_t unit = (uint32_t)(P.block_stride >> 4);
    for (int c = 0; c * kChunk < total; ++c) {
      if (c == kChunks) pdl_wait();   // (from here on it waits for warps that wait there)
      if (c >= kChunks &&
          !__all_sync(0xffffffffu, q4_wait(&page_empty[c % kChunks], ((c / kChunks) & 1) ^ 1, abf, P.wait_ns)))
        break;
      for (int filled = 0; filled < kChunk && have;) {
        const int n = min(kChunk - filled, it.ntiles - ti);
        const int32_t *table = P.block_table + (int64_t)it.b * P.max_blocks;
        int phys[kChunk * kTP / 32];
#pragma unroll
        for (int k = 0; k < kChunk * kTP / 32; ++k) {
          const int e = lane + 32 * k, v = (it.tile0 + ti) * kTP + e;
          // (past the end: the last block once more)
          const int vb = min(v, it.span.nblk - 1);
          phys[k] = e < n * kTP ? table[vb < it.span.nsb ? vb : vb + it.span.skip] : 0;
        }
#pragma unroll
        for (int k = 0; k < kChunk * kTP / 32; ++k) {
          const int e = lane + 32 * k;
          if (e >= n * kTP) continue;
          int ph = phys[k];
          if (ph < 0 || ph >= P.num_blocks) {   // stay in bounds; the output of this sequence is flagged
            bad = true;
            ph = 0;
          }
          const int page = e % kTP;
          s_off[(c % kChunks * kChunk + filled) * kTP + e - page + (page >> 1) + 4 * (page & 1)] = (uint32_t)ph * unit;
        }
        if (lane < n) {
          const int tt = ti + lane;
          s_flag[c % kChunks * kChunk + filled + lane] =
              (tt == 0 ? kFirst : 0) | (tt == it.ntiles - 1 ? kLast | kEnd : 0) | (tt % T == T - 1 ? kEnd : 0) | (tt % T ? kSecond : 0) |
              min(kTP, it.span.nblk - (it.tile0 + tt) * kTP) << 8;
        }
        filled += n;
        ti += n;
        if (ti == it.ntiles) {
          have = q4_next(P, wk, it);
          ti = 0;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&page_full[c % kChunks]);
    }
    pdl_wait();
    if (bad) atomic_or_status(P.status, SV_DEV_BAD_BLOCK);
  } else if (warp == kQWarp) {
    // ------------------------------------------------------------------- Q --
    Q4Walk wk = q4_walk(P, work);
    Q4Item it;
    int i = 0;
    while (q4_next(P, wk, it)) {
      const int buf = i & 1, row = i % 3;
      // the buffer after Q K^T of the item before the last, the rows after the
      // epilogue of the one before that
      bool ok = i < 2 || q4_wait(&q_empty[buf], ((i >> 1) & 1) ^ 1, abf, P.wait_ns);
      if (i >= 3) ok = q4_wait(&o_free[buf ^ 1], ((i - 3) >> 1) & 1, abf, P.wait_ns) && ok;
      if (!__all_sync(0xffffffffu, ok)) break;
      const int64_t ent = (int64_t)it.b * Hp + gp;
      const float *qs = P.ws_qs + ent * (2 * N + 4);
      const float fold = qs[N];
      for (int col = lane; col < N; col += 32) {
        const int w = col / CP, c = col - w * CP;
        const int r = row0 + (c < (w ? rows - live0 : live0) ? w * live0 + c : 0);   // (padding: any)
        const int j = r / P.G;
        s_qs[row][col] = qs[col];
        s_pos[row][col] = j;
        s_row[row][col] = (it.b * P.n_new + j) * P.H_q + g * P.G + (r - j * P.G);
      }
      if (fold < 0.f)
        for (int col = lane; col < N; col += 32) s_qf[row][col] = qs[N + 4 + col];
      if (lane == 0) {
        s_fold[row] = fold;
        s_item[row] = make_int4(it.tile0, it.ntiles, it.span.L, (it.whole ? kWhole : 0) | (it.first ? kOpening : 0));
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive_expect_tx(&q_full[buf], Cfg::kQ);
        bulk_g2s(smem + buf * Cfg::kQ, P.ws_q + ent * Cfg::kQ, Cfg::kQ, &q_full[buf]);
      }
      __syncwarp();
      ++i;
    }
    // the copies in flight land before the CTA may exit
    if (lane == 0)
      for (int k = max(0, i - 2); k < i; ++k)
        if (!mbar_wait(&q_full[k & 1], (k >> 1) & 1)) atomic_or_status(P.status, SV_DEV_TIMEOUT);
  } else if (warp == kQkWarp || warp == kPvWarp) {
    // ----------------------------------------------------------------- MMA --
    // One warp per product; all its lanes wait, one issues. Formats 0 (e4m3 for
    // Q K^T, f16 for P V), f32 accumulators, M = 128.
    constexpr uint32_t idesc_qk = (1u << 4) | ((uint32_t)(N >> 3) << 17) | (8u << 24);
    constexpr uint32_t idesc_pv = idesc_qk | (1u << 16);   // B = P'^T with the rows contiguous
    uint32_t items = 0, step = 0;   // items started, steps done
    bool ok = true;
    if (warp == kQkWarp) {
      for (uint32_t u = 0; u < (uint32_t)total; ++u) {
        const uint32_t bf = u & 1, pb = step & 1;
        pages_of(u, 1, ok);
        const int flag = s_flag[u % (kChunks * kChunk)];
        pages_done(u, 1);
        if (flag & kFirst) {
          ok = q4_wait(&q_full[items & 1], (items >> 1) & 1, abf, P.wait_ns) && ok;
          ++items;
        }
        // the softmax of the step before the last has read the S buffers
        if (!(flag & kSecond) && step >= 2) ok = q4_wait(&p_full[pb], ((step >> 1) & 1) ^ 1, abf, P.wait_ns) && ok;
        ok = q4_wait(&kop_full[bf], (u >> 1) & 1, abf, P.wait_ns) && ok;
        if (!__all_sync(0xffffffffu, ok)) break;
        t5_fence_after();
        if (elect_one()) {
          const uint64_t qd = t5_desc(q_smem + ((items - 1) & 1) * Cfg::kQ, 16, 1024);
          const uint32_t d = tb + Cfg::kSCol + (T * pb + (flag & kSecond ? 1 : 0)) * N, a = tb + Cfg::kKCol + bf * 32;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)   // 32 head dims per MMA, the hi terms of Q and then the lo terms
            t5_mma_ts_f8(d, a + 8 * (kk & 3), qd + (kk >> 2) * (N * 128 / 16) + (kk & 3) * 2, idesc_qk, kk > 0 ? 1u : 0u);
          t5_commit(&kop_empty[bf]);
          if (flag & kEnd) {
            t5_commit(&s_full[pb]);
            mbar_arrive(&s_full[pb]);
          }
          if (flag & kLast) t5_commit(&q_empty[(items - 1) & 1]);
        }
        __syncwarp();
        if (flag & kEnd) ++step;
      }
    } else {
      if (lane < 2) mbar_arrive(&s_full[lane]);   // (no P V before the first steps)
      for (uint32_t u = 0; u < (uint32_t)total; ++u) {
        const uint32_t bf = u & 1, pb = step & 1;
        pages_of(u, 1, ok);
        const int flag = s_flag[u % (kChunks * kChunk)];
        pages_done(u, 1);
        if (flag & kFirst) {
          // O of the item before the last has been read
          if (items >= 2) ok = q4_wait(&o_free[items & 1], ((items >> 1) & 1) ^ 1, abf, P.wait_ns) && ok;
          ++items;
        }
        ok = q4_wait(&vop_full[bf], (u >> 1) & 1, abf, P.wait_ns) && ok;
        if (!(flag & kSecond)) ok = q4_wait(&p_full[pb], (step >> 1) & 1, abf, P.wait_ns) && ok;
        if (!__all_sync(0xffffffffu, ok)) break;
        t5_fence_after();
        if (elect_one()) {
          const uint64_t pd = t5_desc(p_smem + (T * pb + (flag & kSecond ? 1 : 0)) * kPBytes, 16, 1024);
          const uint32_t a = tb + Cfg::kVCol + bf * 64;
          const uint32_t d = tb + Cfg::kOCol + ((items - 1) & 1) * N;
          t5_mma_ts(d, a, pd, idesc_pv, flag & kFirst ? 0u : 1u);   // a block's 16 keys per MMA
          const int nv = flag >> 8;   // blocks past the end have no weight
          if (nv == kTP) {
#pragma unroll
            for (int kk = 1; kk < kTP; ++kk) t5_mma_ts(d, a + 8 * kk, pd + kk * (2048 / 16), idesc_pv, 1u);
          } else {
#pragma unroll 1
            for (int kk = 1; kk < nv; ++kk) t5_mma_ts(d, a + 8 * kk, pd + kk * (2048 / 16), idesc_pv, 1u);
          }
          t5_commit(&vop_empty[bf]);
          if (flag & kEnd) {
            t5_commit(&pv_done[pb]);
            t5_commit(&s_full[pb]);   // the P' buffers are free: part of what the softmax of the step after next waits for
          }
        }
        __syncwarp();
        if (flag & kEnd) ++step;
      }
    }
    // every MMA issued has completed before TMEM can be released
    if (total > 0) {
      uint64_t *dr = &drain[warp - kQkWarp];
      if (elect_one()) t5_commit(dr);
      __syncwarp();
      if (!mbar_wait(dr, 0) && lane == 0) atomic_or_status(P.status, SV_DEV_TIMEOUT);
    }
  } else if (warp >= kKWarp && warp < kPageWarp) {
    // ------------------------------------------------------ codes to TMEM --
    regs_dec<Cfg::kRegsOther>();
    const uint32_t lanes = tb + ((uint32_t)((warp & 3) * 32) << 16);
    auto role = [&](auto is_v) {
      constexpr bool V = decltype(is_v)::value;
      // these four warps take the tiles of one parity, that is, one TMEM buffer
      const uint32_t bf = (warp >> 2) & 1;
      uint64_t *full = (V ? vop_full : kop_full) + bf, *empty = (V ? vop_empty : kop_empty) + bf;
      const uint32_t col = lanes + (V ? Cfg::kVCol + bf * 64 : Cfg::kKCol + bf * 32);
      const int slot = lane & 15, sw = (slot >> 1) & 3;
      // this warp's part of a stage, and of a record
      const uint32_t mine = ring + (warp - kKWarp) * (kNS * 2048);
      const uint8_t *pool = (V ? P.v_cache : P.k_cache) + (int64_t)g * P.head_stride +
                            (V ? (warp & 3) * 256 + (lane & 15) * 16 : lane * 16);
      bool ok = true;
      const uint32_t my_pairs = V ? 0u : pairs + (warp - kKWarp) * (kNS * 256);
      uint32_t fill = 0;   // offset of the next stage to copy to
      auto issue = [&](uint32_t u) {
        if (u < (uint32_t)total) {
          const uint32_t *pg = pages_of(u, 2, ok);
          if (ok) {   // (offsets that never came are not read)
            uint32_t at[4];
            if constexpr (V) {   // 32 head dims of two blocks per copy
              const uint4 a = *reinterpret_cast<const uint4 *>(pg + (lane >> 4) * 4);
              at[0] = a.x; at[1] = a.y; at[2] = a.z; at[3] = a.w;
            } else {             // half a block of keys per copy
              at[0] = at[1] = pg[warp & 3];
              at[2] = at[3] = pg[4 + (warp & 3)];
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
              copy16(mine + fill + lane * 16 + j * 512, pool + (uint64_t)at[j] * 16 + (V ? 0 : (j & 1) * 512));
            if constexpr (!V) {   // the pairs: lanes 0-7 those of the two K blocks, 8-15 of the V blocks
              if (lane < 16)
                copy16(my_pairs + fill / 8 + lane * 16, (lane < 8 ? P.k_cache : P.v_cache) + (int64_t)g * P.head_stride + kCodes +
                                                   (uint64_t)(lane & 4 ? at[2] : at[0]) * 16 + (lane & 3) * 16);
            }
          }
          pages_done(u, 2);
          fill = fill == (kNS - 1) * 2048 ? 0 : fill + 2048;
        }
        copies_commit();
      };
      uint32_t stage = 0;   // offset of the stage to read
      // K: this lane's key in its tile; an odd key, whose V codes come out 16 times
      // too large, has a 16 times smaller weight, and a part 15 that was taken off
      const int key = 32 * (warp & 3) + lane;
      const float shrink = key & 1 ? 0.0625f : 1.f, taken = key & 1 ? 240.f : 0.f;
      const bool run = !(P.withhold & SV_TEST_WITHHOLD_COPIES);
      for (int k = 1 - kNS; run && 2 * k + (int)bf < total; ++k) {   // tile 2 k + bf
        issue(2 * (k + kNS - 1) + bf);
        if (k < 0) continue;
        copies_wait<kNS - 1>();
        __syncwarp();
        if (ok && k > 0) ok = q4_wait(empty, (k & 1) ^ 1, abf, P.wait_ns);
        if (!__all_sync(0xffffffffu, ok)) break;
        t5_fence_after();
        const uint32_t src = mine + stage;
        // (V unrolled by two spills: 127.7 against 122.4 us for 64 sequences)
#pragma unroll (V ? 1 : 2)
        for (int h = 0; h < 4; ++h) {   // K: 32 head dims of a key; V: 32 keys of a head dim
          uint32_t w[4];
          if constexpr (V) {
            uint32_t o[16];
            asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(src + lane * 8 + h * 512));
            asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[2]), "=r"(w[3]) : "r"(src + lane * 8 + h * 512 + 256));
#pragma unroll
            for (int k = 0; k < 4; ++k) spread_v(w[k], o + 4 * k);
            t5_st16(col + 16 * h, o);
          } else {
            uint32_t o[8];
            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                         : "r"(src + lane * 64 + ((h ^ sw) << 4)));
#pragma unroll
            for (int k = 0; k < 4; ++k) spread_k(w[k], o + 2 * k);
            t5_st8(col + 8 * h, o);
          }
        }
        if constexpr (!V) {
          uint32_t kp, vp;
          asm volatile("ld.shared.u32 %0, [%1];" : "=r"(kp) : "r"(my_pairs + stage / 8 + lane * 4));
          asm volatile("ld.shared.u32 %0, [%1];" : "=r"(vp) : "r"(my_pairs + stage / 8 + lane * 4 + 128));
          const float2 k2 = __half22float2(*reinterpret_cast<const __half2 *>(&kp));
          const float2 v2 = __half22float2(*reinterpret_cast<const __half2 *>(&vp));
          const float vs = fmaxf(v2.x, 5.9604645e-8f) * shrink;   // (pages never written hold zeros)
          const float vi = rcpf(vs), vz = fmaf(v2.y, vi, taken);
          const uint32_t dst = scales + (uint32_t)(2 * k + bf) % kScales * kScaleBytes;
          asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(dst + key * 16), "f"(k2.x), "f"(k2.y * P.scale_log2),
                       "f"(lg2f(vs)), "f"(vi)
                       : "memory");
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(dst + kTK * 16 + key * 4), "f"(vz) : "memory");
        }
        t5_wait_st();
        t5_fence_before();
        stage = stage == (kNS - 1) * 2048 ? 0 : stage + 2048;
        __syncwarp();   // (every lane has read its codes: the stage is refilled next)
        if (lane == 0) mbar_arrive(full);
      }
      copies_wait<0>();
    };
    if (warp >= kVWarp) role(std::true_type{});
    else role(std::false_type{});
  } else if (warp < softmax_warps) {
    // ------------------------------------------------------------- softmax --
    regs_inc<Cfg::kRegsSoftmax>();
    const int w = warp >> 2, t = tid & 127;
    const int c_first = w * CP;                 // this warpgroup's columns
    const int live = w ? rows - live0 : live0;
    const int bar = 1 + w;
    const uint32_t lanes = tb + ((uint32_t)((warp & 3) * 32) << 16);
    // row of P' that this thread's key takes (the order of the codes)
    const int prow = (t & ~7) | ((t & 3) << 1) | ((t >> 2) & 1);
    const uint32_t sign = t & 1 ? 0x80008000u : 0u;   // odd keys' weights are negative
    int u = 0, i = 0;            // tiles and items done
    uint32_t step = 0;
    // A wait that gave up (ok false) only shows at the warpgroup's next vote, so
    // that its four warps leave together.
    bool ok = true;
    // The epilogue's second part, a head dim per thread: O of an item, once its
    // last P V is done; it is taken after the next item's first step, which hides
    // that P V.
    struct { bool pending, whole; uint32_t step; int i; int64_t ent; } done = {false, false, 0, 0, 0};
    auto finish = [&] {
      done.pending = false;
      ok = __all_sync(0xffffffffu, q4_wait(&pv_done[done.step & 1], (done.step >> 1) & 1, abf, P.wait_ns)) && ok;
      if (!ok) return;
      t5_fence_after();
      float o[NC];
      t5_ldn(lanes + Cfg::kOCol + (done.i & 1) * N + c_first, reinterpret_cast<uint32_t(&)[NC]>(o));
      t5_wait_ld();
      keep_after<NC>(o);
#pragma unroll
      for (int k = 0; k < NC; ++k) {
        if (k >= live) break;
        const float2 f = s_fin[done.i & 1][c_first + k];
        const float x = fmaf(o[k], 0x1p24f, f.y) * f.x;
        if (done.whole)
          static_cast<__nv_bfloat16 *>(P.out)[(int64_t)s_row[done.i % 3][c_first + k] * kD + t] = __float2bfloat16_rn(x);
        else
          P.ws_acc[(done.ent * P.Rg + w * live0 + k) * kD + t] = x;
      }
      t5_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_free[done.i & 1]);
    };
    while (u < total) {
      const int buf = i % 3;
      const uint32_t o_col = lanes + Cfg::kOCol + (i & 1) * N + c_first;
      ok = __all_sync(0xffffffffu, q4_wait(&q_full[i & 1], (i >> 1) & 1, abf, P.wait_ns)) && ok;
      const float fold = P.scale_log2 * s_fold[buf];
      const int4 it = s_item[buf];
      const int tile0 = it.x, ntiles = it.y, L = it.z;
      const int edge0 = fold < 0.f ? INT_MIN : L - P.n_new - T * kTK + 2, edge1 = P.window > 0 ? L - P.window : 0;
      if (t < NC) s_nb[c_first + t] = 0.f;
      float2 l2[NC / 2], b2[NC / 2];
#pragma unroll
      for (int k = 0; k < NC / 2; ++k) l2[k] = b2[k] = make_float2(0.f, 0.f);
      bool gone = bar_or(bar, 128, !ok);
      for (int ti = 0; ti < ntiles && !gone; ++step) {
        const int nt = min(ntiles - ti, T);
        // S of this step, and with it the keys' scales and P' buffers that P V two
        // steps ago has read
        const int pb = step & 1;
        ok = q4_wait(&s_full[pb], (step >> 1) & 1, abf, P.wait_ns) && ok;
        float ka[T], kb[T], vc[T], vi[T], vz[T];
#pragma unroll
        for (int h = 0; h < T; ++h) {   // this thread's keys
          const uint32_t src = scales + (uint32_t)(u + h) % kScales * kScaleBytes;
          asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(ka[h]), "=f"(kb[h]), "=f"(vc[h]), "=f"(vi[h]) : "r"(src + t * 16));
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(vz[h]) : "r"(src + kTK * 16 + t * 4));
          ka[h] *= fabsf(fold);
        }
        const uint32_t s_col = lanes + Cfg::kSCol + T * pb * N + c_first;
        // A step that ends past the oldest query or holds keys that a window has
        // left: position j sees a key iff 0 <= j - j0 < reach. A key that no
        // position sees (past the end, or between sinks and window) may hold
        // anything.
        const int key0 = (tile0 + ti) * kTK;
        const bool edge = key0 >= edge0 || key0 < edge1;
        int j0[T] = {};
        uint32_t reach[T] = {};
        if (edge) {
#pragma unroll
          for (int h = 0; h < T; ++h) {
            const int key = key0 + h * kTK + t;
            j0[h] = key - (L - P.n_new);
            reach[h] = P.window > 0 && key >= P.sinks ? (uint32_t)P.window : 0x80000000u;
            if (key >= L || (uint32_t)(P.n_new - 1 - j0[h]) >= reach[h] + (uint32_t)(P.n_new - 1)) vi[h] = vz[h] = 0.f;
          }
          // Rows with powers of their own (every step of such an item counts as
          // an edge: a test apart, a second copy of the steps or a factor a score
          // cost every call 3 to 7 %; this way it is 64 sequences 126.9 against
          // 123.5 us, and 180 us where rows do have them).
          ok = __all_sync(0xffffffffu, ok);
          if (fold < 0.f && ok) q4_scale_rows<NC, N>(s_col, nt, &s_qf[buf][c_first]);
        }
        ok = __all_sync(0xffffffffu, ok);
        t5_fence_after();
        float2 y[T][NC / 2];   // log2 weights, minus the reference
        auto scores = [&](int h) {
          const float2 ka2 = make_float2(ka[h], ka[h]), kb2 = make_float2(kb[h], kb[h]), vc2 = make_float2(vc[h], vc[h]);
          uint32_t x[NC];
          t5_ldn(s_col + h * N, x);
          t5_wait_ld();
#pragma unroll
          for (int k = 0; k < NC; k += 4) {
            const float4 qs = *reinterpret_cast<const float4 *>(&s_qs[buf][c_first + k]);
            const float4 nb = *reinterpret_cast<const float4 *>(&s_nb[c_first + k]);
            const float2 z0 = __ffma2_rn(make_float2(qs.x, qs.y), kb2, __fadd2_rn(vc2, make_float2(nb.x, nb.y)));
            const float2 z1 = __ffma2_rn(make_float2(qs.z, qs.w), kb2, __fadd2_rn(vc2, make_float2(nb.z, nb.w)));
            y[h][k / 2] = __ffma2_rn(make_float2(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), ka2, z0);
            y[h][k / 2 + 1] = __ffma2_rn(make_float2(__uint_as_float(x[k + 2]), __uint_as_float(x[k + 3])), ka2, z1);
          }
          if (edge) {
#pragma unroll
            for (int k = 0; k < NC; k += 4) {
              const int4 j = *reinterpret_cast<const int4 *>(&s_pos[buf][c_first + k]);
              if ((uint32_t)(j.x - j0[h]) >= reach[h]) y[h][k / 2].x = -INFINITY;
              if ((uint32_t)(j.y - j0[h]) >= reach[h]) y[h][k / 2].y = -INFINITY;
              if ((uint32_t)(j.z - j0[h]) >= reach[h]) y[h][k / 2 + 1].x = -INFINITY;
              if ((uint32_t)(j.w - j0[h]) >= reach[h]) y[h][k / 2 + 1].y = -INFINITY;
            }
          }
        };
        const bool first = ti == 0;
        for (int again = 0;; ++again) {
          scores(0);
          if constexpr (T > 1) {
            if (nt > 1) {
              scores(1);
            } else {
#pragma unroll
              for (int k = 0; k < NC / 2; ++k) y[1][k] = make_float2(-INFINITY, -INFINITY);
            }
          }
          if (again) break;
          // The first step of a sequence sets the references (they are 0 so
          // far); later ones move when a weight exceeds 2^kMove. All four warps
          // decide together, as they share O.
          float top = fmaxf(y[0][0].x, y[0][0].y);
#pragma unroll
          for (int k = 1; k < NC / 2; ++k) top = fmaxf(fmaxf(top, y[0][k].x), y[0][k].y);
          if constexpr (T > 1) {
#pragma unroll
            for (int k = 0; k < NC / 2; ++k) top = fmaxf(fmaxf(top, y[1][k].x), y[1][k].y);
          }
          if (!bar_or(bar, 128, first || top > kMove || !ok)) break;
          if (bar_or(bar, 128, !ok)) {
            gone = true;
            break;
          }
          // each column's largest weight, without the reference
          if (first) {
            float mine = -INFINITY;
#pragma unroll
            for (int k = 0; k < NC; ++k) {
              const float m = warp_top(k & 1 ? fmaxf(y[0][k / 2].y, y[T - 1][k / 2].y) : fmaxf(y[0][k / 2].x, y[T - 1][k / 2].x));
              if (lane == k) mine = m;
            }
            if (lane < NC) s_max[warp][lane] = mine;
          } else {
#pragma unroll 1
            for (int k = 0; k < live; ++k) {
              float m = -INFINITY;
#pragma unroll
              for (int h = 0; h < T; ++h) {
                if (h >= nt) break;
                uint32_t xs;
                asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(xs) : "r"(s_col + h * N + k));
                t5_wait_ld();
                const float z = fmaf(__uint_as_float(xs), ka[h], fmaf(s_qs[buf][c_first + k], kb[h], vc[h]));
                if (!edge || (uint32_t)(s_pos[buf][c_first + k] - j0[h]) < reach[h]) m = fmaxf(m, z);
              }
              m = warp_max(m);
              if (lane == 0) s_max[warp][k] = m;
            }
          }
          named_bar_sync(bar, 128);
          if (t < NC) {
            float a = 1.f, nb = first ? kUnset : s_nb[c_first + t];
            if (t < live) {
              const float m = fmaxf(fmaxf(s_max[4 * w][t], s_max[4 * w + 1][t]), fmaxf(s_max[4 * w + 2][t], s_max[4 * w + 3][t]));
              if (m + nb > kMove) {   // (a row that has met no key keeps kUnset)
                a = ex2f(kTop - m - nb);
                nb = kTop - m;
              }
            } else {
              nb = -kUnset;   // padding never moves
            }
            s_nb[c_first + t] = nb;
            s_a[c_first + t] = a;
          }
          named_bar_sync(bar, 128);
          if (first) {
#pragma unroll
            for (int k = 0; k < NC; k += 4) {
              const float4 nb = *reinterpret_cast<const float4 *>(&s_nb[c_first + k]);
#pragma unroll
              for (int h = 0; h < T; ++h) {
                y[h][k / 2] = __fadd2_rn(y[h][k / 2], make_float2(nb.x, nb.y));
                y[h][k / 2 + 1] = __fadd2_rn(y[h][k / 2 + 1], make_float2(nb.z, nb.w));
              }
            }
            break;
          } else {
#pragma unroll
            for (int k = 0; k < NC; k += 4) {
              const float4 a = *reinterpret_cast<const float4 *>(&s_a[c_first + k]);
              l2[k / 2] = __fmul2_rn(l2[k / 2], make_float2(a.x, a.y));
              b2[k / 2] = __fmul2_rn(b2[k / 2], make_float2(a.x, a.y));
              l2[k / 2 + 1] = __fmul2_rn(l2[k / 2 + 1], make_float2(a.z, a.w));
              b2[k / 2 + 1] = __fmul2_rn(b2[k / 2 + 1], make_float2(a.z, a.w));
            }
            // O too, once the previous P V has landed
            ok = __all_sync(0xffffffffu, q4_wait(&pv_done[pb ^ 1], ((step - 1) >> 1) & 1, abf, P.wait_ns)) && ok;
            t5_fence_after();
#pragma unroll 1
            for (int k = 0; k < live; ++k) {
              uint32_t o;
              const uint32_t at = o_col + k;
              asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(o) : "r"(at));
              t5_wait_ld();
              o = __float_as_uint(__uint_as_float(o) * s_a[c_first + k]);
              asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(at), "r"(o) : "memory");
            }
            t5_wait_st();
          }
        }
        if (gone) break;
        const uint32_t p_row = p_smem + T * pb * kPBytes + prow * 128;
#pragma unroll
        for (int h = 0; h < T; ++h) {
          if (h >= nt) break;
          const float2 vi2 = make_float2(vi[h], vi[h]), vz2 = make_float2(vz[h], vz[h]);
#pragma unroll
          for (int c = 0; c < NC; c += 8) {
            uint32_t ph[4];
#pragma unroll
            for (int k = 0; k < (NC - c < 8 ? 2 : 4); ++k) {
              const int e = c / 2 + k;
              const float2 p = make_float2(ex2f(y[h][e].x), ex2f(y[h][e].y));
              l2[e] = __ffma2_rn(p, vi2, l2[e]);
              b2[e] = __ffma2_rn(p, vz2, b2[e]);
              ph[k] = pack2<true>(p.x, p.y) ^ sign;
            }
            const uint32_t dst = p_row + h * kPBytes + ((((c_first + c) >> 3) ^ (prow & 7)) << 4);
            if (NC - c < 8)   // (what the columns of padding hold does not matter)
              asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(dst), "r"(ph[0]), "r"(ph[1]) : "memory");
            else
              asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(dst), "r"(ph[0]), "r"(ph[1]), "r"(ph[2]), "r"(ph[3])
                           : "memory");
          }
        }
        fence_proxy_async_shared();
        t5_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[pb]);
        ti += nt;
        u += nt;
        if (done.pending) finish();
      }
      if (gone) break;
      // ---- epilogue, first part: sums over the keys -------------------------
      {
        float v[2 * NC];
#pragma unroll
        for (int k = 0; k < NC; ++k) {
          v[k] = k & 1 ? l2[k / 2].y : l2[k / 2].x;
          v[NC + k] = k & 1 ? b2[k / 2].y : b2[k / 2].x;
        }
        int at = 0, n = 0;
        warp_sums<2 * NC>(v, lane, at, n);
#pragma unroll
        for (int k = 0; k < 5; ++k)   // (lanes with the same sums write the same words)
          if (k < n) s_red[warp][at + k] = v[k];
      }
      named_bar_sync(bar, 128);
      const int64_t ent = 2 * (int64_t)blockIdx.x + (it.w & kOpening ? 0 : 1);
      if (t < live) {
        float l = 0.f, b = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          l += s_red[4 * w + k][t];
          b += s_red[4 * w + k][NC + t];
        }
        // (a row of NaN stays NaN; l is 0 only for a row without keys, which a query that sees itself never is)
        s_fin[i & 1][c_first + t] = make_float2(it.w & kWhole ? 1.f / l : 1.f, b);
        if (!(it.w & kWhole)) {
          const int64_t e = ent * P.Rg + w * live0 + t;
          P.ws_ml[2 * e] = -s_nb[c_first + t];
          P.ws_ml[2 * e + 1] = l;
        }
      }
      done = {true, (it.w & kWhole) != 0, step - 1, i, ent};
      ++i;
    }
    named_bar_sync(bar, 128);
    if (done.pending) finish();
  }
  __syncthreads();
  if (tid == 0 && *abf) atomic_or_status(P.status, SV_DEV_TIMEOUT);
  t5_fence_after();
  if (warp == kQkWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tb), "r"(512));
}

// Merge of the sequences that more than one range holds: CTA (range r, kv head
// and row group, eight rows) leaves at once unless r's start is the first cut
// of a sequence. Its pieces come from ranges r - 1 (the last item of its CTA,
// or the first if that range starts with the sequence), r, r + 1, ... (first
// items); a warp takes a row, lane l the head dims 4l .. 4l + 3, and loads
// eight pieces at once.
constexpr int kMergeWarps = 8;
__global__ void __launch_bounds__(32 * kMergeWarps) attn_q4_merge_kernel(const __grid_constant__ Q4Params P) {
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

int q4_sms() {
  static int n = 0;
  static std::once_flag once;
  std::call_once(once, [] {
    int dev = 0;
    cudaGetDevice(&dev);
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) n = 148;
  });
  return n;
}

struct Q4Plan {
  bool tc;
  int R, RG, Rg, NR, C;
};

Q4Plan q4_plan(int B, int n_new, int H_q, int H_kv, int d, int max_blocks, int bs, sv_dtype qd, int window, int sinks) {
  Q4Plan p = {};
  const int span = span_blocks_max(max_blocks, n_new, window, sinks, bs);
  const int64_t tiles = (int64_t)std::max(B, 1) * ((span + kTP - 1) / kTP);
  const int64_t R = (int64_t)n_new * (H_q / H_kv);
  p.tc = qd == SV_BF16 && d == kD && bs == kBS && R <= 128 && tiles < (1ll << 30) &&
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
  p.NR = tiles <= 4 ? 1 : (int)std::max<int64_t>(1, std::min<int64_t>(q4_sms() / Hp, tiles));
  p.C = (int)(p.NR * Hp);
  return p;
}

// Columns of S and O, a softmax warpgroup's rows in steps of 4 (of 8 for the layout)
int q4_cols(const Q4Plan &p) { return 2 * ((q4_first(p.Rg) + 7) / 8 * 8); }

size_t q4_ws_bytes(const Q4Plan &p, int B, int H_kv) {
  const size_t ent = (size_t)2 * p.C * p.Rg, qent = (size_t)B * H_kv * p.RG, n = q4_cols(p);
  return align_up(ent * kD * sizeof(float), 256) + align_up(ent * 2 * sizeof(float), 256) +
         align_up((size_t)p.NR * sizeof(int4), 256) + align_up(qent * n * 256, 256) +
         align_up(qent * (2 * n + 4) * sizeof(float), 256);
}

template <int NC>
sv_status launch_q4(const Q4Params &P, int C, cudaStream_t st) {
  static DeviceOnce once;
  const cudaError_t err = once_per_device(once, [] {
    return cudaFuncSetAttribute(attn_q4_kernel<NC>, cudaFuncAttributeMaxDynamicSharedMemorySize, Q4Cfg<NC>::kSmem);
  });
  if (err != cudaSuccess) return fail(SV_ERR_CUDA, "spec_verify_attn_q4: cudaFuncSetAttribute: %s", cudaGetErrorString(err));
  const int64_t prep = (P.NR + kPrepWarps - 1) / kPrepWarps + (int64_t)P.B * P.H_kv * P.RG;
  launch_k(attn_q4_prep_kernel<NC>, dim3((unsigned)prep), dim3(32 * kPrepWarps), 0, st, 1, P);
  launch_k(attn_q4_kernel<NC>, dim3(C), dim3(32 * kWarps), Q4Cfg<NC>::kSmem, st, 1, P);
  return check_launch("spec_verify_attn_q4 launch");
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" size_t spec_verify_attn_q4_workspace_size(int B, int n_new, int H_q, int H_kv, int d_head,
                                                     int max_blocks_per_seq, int block_size, int window, int sinks) {
  const size_t other = spec_verify_attn_window_workspace_size(B, n_new, H_q, H_kv, d_head, max_blocks_per_seq,
                                                              block_size, window, sinks);
  if (other == 0) return 0;
  if ((int64_t)window >= (int64_t)max_blocks_per_seq * block_size) window = sinks = 0;
  const Q4Plan p = q4_plan(B, n_new, H_q, H_kv, d_head, max_blocks_per_seq, block_size, SV_BF16, window, sinks);
  // (queries in f32 run on the CUDA-core kernel whatever the shape)
  return p.tc ? std::max(other, q4_ws_bytes(p, B, H_kv)) : other;
}

extern "C" sv_status spec_verify_attn_q4(const void *q, sv_dtype q_dtype, const void *k_cache, const void *v_cache,
                                         const sv_kv_layout *layout, const int32_t *block_table,
                                         int max_blocks_per_seq, const int32_t *seq_lens, int B, int n_new, int H_q,
                                         int H_kv, int d_head, int block_size, int num_blocks, float softmax_scale,
                                         int window, int sinks, void *out, sv_dtype out_dtype, void *workspace,
                                         size_t workspace_bytes, int32_t *dev_status, sv_stream_t stream) {
  if (window < 0 || sinks < 0) return fail(SV_ERR_INVALID_ARG, "spec_verify_attn_q4: negative window or sinks");
  if (max_blocks_per_seq > 0 && block_size > 0 && !capacity_ok(max_blocks_per_seq, block_size))
    return fail(SV_ERR_UNSUPPORTED, "spec_verify_attn_q4: max_blocks_per_seq * block_size must be below 2^30");
  Q4Plan p = {};
  const bool sizes_ok = B >= 0 && n_new >= 1 && H_q >= 1 && H_kv >= 1 && H_q % H_kv == 0 && num_blocks >= 1 &&
                        max_blocks_per_seq >= 1 && H_kv <= 65535 && block_size >= 1;
  int win = window, snk = sinks;
  if ((int64_t)win >= (int64_t)max_blocks_per_seq * block_size) win = snk = 0;   // reaches every key
  // (block offsets are held in 32 bits, in 16-byte units)
  const int64_t bstride = layout ? layout->block_stride : (int64_t)q4_record_bytes(kD, kBS) * H_kv;
  if (sizes_ok && (int64_t)num_blocks * (bstride / 16) < (1ll << 32)) p = q4_plan(B, n_new, H_q, H_kv, d_head, max_blocks_per_seq, block_size, q_dtype, win, snk);
  if (!p.tc || q_dtype != out_dtype)
    return attn_cuda_core_q4(q, q_dtype, k_cache, v_cache, layout, block_table, max_blocks_per_seq, seq_lens, B, n_new,
                             H_q, H_kv, d_head, block_size, num_blocks, softmax_scale, window, sinks, out, out_dtype,
                             workspace, workspace_bytes, dev_status, stream);
  if (!q || !k_cache || !v_cache || !block_table || !seq_lens || !out)
    return fail(SV_ERR_INVALID_ARG, "spec_verify_attn_q4: null pointer argument");
  if (!(softmax_scale > 0.f) || !std::isfinite(softmax_scale))
    return fail(SV_ERR_INVALID_ARG, "spec_verify_attn_q4: softmax_scale must be finite and > 0");
  Q4Params P;
  memset(&P, 0, sizeof(P));
  const sv_status rc = q4_check("spec_verify_attn_q4", k_cache, v_cache, layout, H_kv, d_head, block_size,
                                &P.block_stride, &P.head_stride);
  if (rc != SV_OK) return rc;
  const size_t need = q4_ws_bytes(p, B, H_kv);
  if (!workspace || workspace_bytes < need)
    return fail(SV_ERR_WORKSPACE, "spec_verify_attn_q4: workspace needs %zu bytes", need);
  if (!aligned(workspace, 256)) return fail(SV_ERR_WORKSPACE, "spec_verify_attn_q4: workspace not 256-byte aligned");
  if (!aligned(q, 16) || !aligned(out, 16))
    return fail(SV_ERR_INVALID_ARG, "spec_verify_attn_q4: q and out must be 16-byte aligned");
  if (B == 0) return ok();
  const size_t ent = (size_t)2 * p.C * p.Rg;
  P.q = q; P.out = out;
  P.k_cache = static_cast<const uint8_t *>(k_cache); P.v_cache = static_cast<const uint8_t *>(v_cache);
  P.block_table = block_table; P.seq_lens = seq_lens;
  P.ws_acc = static_cast<float *>(workspace);
  P.ws_ml = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + align_up(ent * kD * sizeof(float), 256));
  uint8_t *at = reinterpret_cast<uint8_t *>(P.ws_ml) + align_up(ent * 2 * sizeof(float), 256);
  P.ws_split = reinterpret_cast<int4 *>(at);
  at += align_up((size_t)p.NR * sizeof(int4), 256);
  P.ws_q = at;
  at += align_up((size_t)B * H_kv * p.RG * q4_cols(p) * 256, 256);
  P.ws_qs = reinterpret_cast<float *>(at);
  P.status = dev_status;
  P.B = B; P.n_new = n_new; P.H_q = H_q; P.H_kv = H_kv; P.G = H_q / H_kv; P.R = p.R; P.Rg = p.Rg; P.RG = p.RG;
  P.NR = p.NR; P.max_blocks = max_blocks_per_seq; P.num_blocks = num_blocks; P.window = win; P.sinks = snk;
  P.scale_log2 = (float)((double)softmax_scale * 1.4426950408889634074);
  P.wait_ns = wait_limit_ns();
  P.withhold = test_withhold();
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int half = q4_first(p.Rg);   // rows of a softmax warpgroup
  const sv_status r2 = half <= 4    ? launch_q4<4>(P, p.C, st)
                       : half <= 8  ? launch_q4<8>(P, p.C, st)
                       : half <= 12 ? launch_q4<12>(P, p.C, st)
                       : half <= 16 ? launch_q4<16>(P, p.C, st)
                       : half <= 20 ? launch_q4<20>(P, p.C, st)
                       : half <= 24 ? launch_q4<24>(P, p.C, st)
                                    : launch_q4<32>(P, p.C, st);
  if (r2 != SV_OK || p.NR == 1) return r2;
  launch_k(attn_q4_merge_kernel, dim3((p.NR - 1) * H_kv * p.RG, (p.Rg + kMergeWarps - 1) / kMergeWarps),
           dim3(32 * kMergeWarps), 0, st, 1, P);
  return check_launch("spec_verify_attn_q4 merge launch");
}
