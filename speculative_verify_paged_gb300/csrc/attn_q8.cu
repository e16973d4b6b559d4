// spec_verify_attn_q8: paged GQA verify attention over an 8-bit block-scaled
// cache (page layout: q8.cuh), on the tensor cores for d_head 128, 16-token
// blocks and bf16 queries.
//
// Mathematics. With K_t = s_t c_t and V_t = s'_t c'_t (c, c' e4m3 codes, one scale
// per block), for query row r
//   x_rt = scale s_t (q_r . c_t),
//   p'_rt = s'_t 2^(x_rt - ref_r)            (log2 domain, ref_r a running reference)
//   out_r = sum_t p'_rt c'_t / sum_t (p'_rt / s'_t)
// so both products run on the codes as they lie in the pages, and the scales enter
// per key.
//
// Operands. Codes go from the pages to shared memory by tensor copies (a block of
// a kv head is 16 rows of 128 bytes) and from there to the tensor cores: nothing
// is unpacked. Q K^T takes each query row as two e4m3 terms (hi + lo, kl_prep_kernel).
// P V has e4m3 codes on one side, so the weights have to be 8-bit too, and e4m3
// would not do: the sum over a long row needs the small weights as well. A weight
// is rounded to f16 and cut into three e5m2 terms, which is a matter of bytes: the
// upper byte of an f16 is an e5m2 number, what is left after taking the nearest off is
// exact in f16 again, and so on; the third is taken 32 times (cut_weights). From 2^-10
// on the terms hold the f16 exactly, so such weights keep f16's 2^-11; below, they are
// off by at most 2^-21, and f16's subnormals by 2^-25. A row's largest weight is at
// least 2^kTop: 2^-11 relative down to 2^-15 of the largest, and 2^-25 of it below.
// kind::f8f6f4 takes e4m3 and e5m2 side by side.
// Keys on the lanes: S^T = C Q^T, O^T = C'^T P'^T (key_lanes.cuh). C is K-major as
// it lies, C'^T is read across its rows (head dims contiguous), P' is written by
// the key's thread as a row of its columns.
//
// What bounds it. Up to 16 query rows a kv head, memory: 64 sequences of 8192 keys,
// 1.07 GB, 174 to 177 us with 4 to 16 rows. Above, the chain of a softmax step (scores from
// tensor memory, the vote on the references, powers, terms, their way to shared
// memory), which W warpgroups take side by side: at 64 sequences of 4750 keys and 40
// rows a tile costs 1710 cycles, 1290 of them what its bytes take; the schedulers
// issue in two thirds, and with nearly no products it would be a tenth faster. What
// got it there, at 64 sequences of 1024 .. 8192 keys, 40 rows, 616 MB: references
// moved in registers instead of from tensor memory 319 -> 177 us; the terms as columns
// of one wide product, the scales by a warp of their own 161; eight rows a warpgroup
// 153; edge flags with the scales and little else carried along 144; five warpgroups
// with 80 registers instead of six with 72 134; fixed addresses of the terms 132; and
// the terms rounded instead of cut off cost 2. Some 15 us of it, and all of a short
// single call's 17, are the three launches and the way from a page's number to its
// first score.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>
#include <type_traits>

#include "key_lanes.cuh"
#include "q8.cuh"

namespace sv {
namespace {

constexpr int kTile = kTK * kD;            // bytes of a tile of K or V
constexpr int kEdge = 16;                  // of a tile: some query does not see all its keys
// A row's reference puts its largest weight at 2^kTop and moves once one exceeds
// 2^kMove (rounded to f16 that is 61152, the nearest e5m2 to which is its largest, 57344).
constexpr float kTop = 5.f, kMove = 15.9f;

template <int NC, int W> struct Q8Cfg : KlCfg<NC, W> {
  using KlCfg<NC, W>::kN;
  using KlCfg<NC, W>::kQ;
  using KlCfg<NC, W>::kT;
  // Registers a thread: at the launch, of the softmax warps, which take what the
  // others leave, and of those.
  static constexpr int kWarps = 4 * W + 8;
  static constexpr int kRegs = W == 2 ? 128 : W == 4 ? 80 : W == 5 ? 72 : 64;
  static constexpr int kRegsSoftmax = W == 2 ? 192 : W == 4 ? 96 : W == 5 ? 80 : 72, kRegsOther = W == 2 ? 64 : W <= 5 ? 48 : 40;
  static_assert(4 * W * kRegsSoftmax + 8 * kRegsOther <= kWarps * kRegs, "registers");
  // The terms of P', and where tensor memory has room those of Q, side by side are
  // the columns of one product with several sums: what an MMA of few columns costs
  // is its other operand, 4 KB from shared memory (16 or 32 columns 41 cycles, 48 45,
  // 96 57, 144 72).
  static constexpr int kSSums = kN <= 32 ? 2 : 1, kSCols = kSSums * kN, kOCols = 3 * kN;
  // P' lies in atoms of 32 columns, 32 bytes a key.
  static constexpr int kAtom = kTK * 32, kPBytes = (kOCols + 31) / 32 * kAtom;
  static constexpr int kStatic = 7680 + 80 * kN;                   // static shared memory, at most
  static constexpr int kFixed = 1024 + 2 * kQ + 2 * kT * kPBytes;
  static constexpr int kAll = (227 * 1024 - kStatic - kFixed) / kTile;   // stages that fit
  static constexpr int kVS = (kAll + 1) / 2 < 5 ? (kAll + 1) / 2 : 5, kKS = kAll - kVS < 5 ? kAll - kVS : 5;
  static constexpr int kSmem = kFixed + (kKS + kVS) * kTile;
  static constexpr uint32_t kSCol = 0, kOCol = 2 * kT * kSCols;   // (two buffers each)
  static_assert(kOCol + 2 * kOCols <= 512, "TMEM columns");
  static_assert(kKS >= 2 && kVS >= 2, "shared memory");
};

struct Q8Maps {
  CUtensorMap k, v;   // {head dim, slot, kv head, block}, boxes of 128 x 16
};

template <int R> __device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R> __device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }

// A shared-memory operand in atoms of 32 bytes by 8 rows, `lbo` apart along the
// 32 bytes and `sbo` along the rows.
__device__ __forceinline__ uint64_t t5_desc32(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFF);
  d |= (uint64_t)((lbo >> 4) & 0x3FFF) << 16;
  d |= (uint64_t)((sbo >> 4) & 0x3FFF) << 32;
  d |= (uint64_t)1 << 46;   // descriptor version of the sm_100 family
  d |= (uint64_t)6 << 61;   // 32-byte swizzle
  return d;
}

// Four weights (two f16 pairs) as three words of e5m2, each term the nearest to what
// is left: half a step added to the bits moves a magnitude to the nearest upper byte
// (below 2^16 none becomes an infinity), and what it then exceeds or leaves, of
// either sign, is exact in f16. Of an f16's ten bits after the first the first term
// leaves at most the lower seven, the second the lower three, which the third, 32 times,
// holds. (Terms cut off instead of rounded would leave up to 2^-9, and on average more
// than nothing.) NaN becomes zeros: the row's sum carries it.
constexpr float kCut = 0.03125f;
__device__ __forceinline__ void cut_weights(uint32_t h0, uint32_t h1, uint32_t (&w)[3]) {
  auto near = [](uint32_t h) { return h + 0x00800080u; };   // (no NaN but 0x7fff: no carry into the other half)
  auto rest = [](uint32_t h, uint32_t n) {   // minus the term's value
    const uint32_t u = n & 0xFF00FF00u;
    const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&h), *reinterpret_cast<const __half2 *>(&u));
    return *reinterpret_cast<const uint32_t *>(&r);
  };
  auto last = [](uint32_t h) {
    const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&h), __float2half2_rn(32.f));
    return *reinterpret_cast<const uint32_t *>(&r) + 0x00800080u;
  };
  uint32_t n0 = near(h0), n1 = near(h1);
  w[0] = __byte_perm(n0, n1, 0x7531);
  h0 = rest(h0, n0);
  h1 = rest(h1, n1);
  n0 = near(h0);
  n1 = near(h1);
  w[1] = __byte_perm(n0, n1, 0x7531);
  w[2] = __byte_perm(last(rest(h0, n0)), last(rest(h1, n1)), 0x7531);
}

// W warpgroups: softmax (a key per thread and tile; each warpgroup its share of
// the query rows, or the first all of up to 8), later the epilogue (a head dim
// per thread). Then eight warps: block numbers and flags of the tiles ahead; copies
// of the K codes; of the V codes; Q K^T, which owns the 512 TMEM columns; P V; Q of
// the next sequence; the blocks' scales; one idle.
template <int NC, int W>
__global__ void __launch_bounds__(32 * Q8Cfg<NC, W>::kWarps, 1) attn_q8_kernel(const __grid_constant__ KlParams P, const __grid_constant__ Q8Maps M) {
  using Cfg = Q8Cfg<NC, W>;
  constexpr int kPageWarp = 4 * W, kKWarp = kPageWarp + 1, kVWarp = kPageWarp + 2, kQkWarp = kPageWarp + 3, kPvWarp = kPageWarp + 4,
                kQWarp = kPageWarp + 5, kScaleWarp = kPageWarp + 6;
  constexpr int N = Cfg::kN, CP = Cfg::kCols, T = Cfg::kT, KS = Cfg::kKS, VS = Cfg::kVS;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t page_full[kChunks], page_empty[kChunks], scale_full[kChunks];
  __shared__ int s_phys[kChunks * kChunk * kTP];   // blocks of the tiles ahead
  __shared__ __align__(16) float4 s_scale[kChunks * kChunk * kTP];   // their scales: of K, log2 of V's, 1 / V's; not 0 in an edge tile
  __shared__ int s_flag[kChunks * kChunk];   // kFirst, kLast, kEnd, kSecond, kEdge, blocks of the tile << 8
  // rows of V that no query sees: [z0, z1) and from z2 on, z0 | z1 << 8 | z2 << 16
  __shared__ int s_zero[kChunks * kChunk];
  __shared__ __align__(8) uint64_t k_full[KS], k_empty[KS], v_full[VS], v_empty[VS];
  __shared__ __align__(8) uint64_t s_full[2], p_full[2], pv_done[2], q_full[2], q_empty[2], o_free[2], drain[2];
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  __shared__ int4 s_work;
  // per row of the items in flight: position (0 .. n_new - 1), row of q and out, its own power of two; per item the
  // power of two that undoes Q's scaling (-1: the rows have their own)
  __shared__ __align__(16) float s_qf[3][N];
  __shared__ __align__(16) int s_pos[3][N];
  __shared__ int s_row[3][N];
  __shared__ float s_fold[3];
  __shared__ __align__(16) int4 s_item[3];   // first tile, tiles, length in span coordinates, kWhole | kOpening
  __shared__ __align__(16) float s_nb[N], s_by[N], s_a[N];   // minus the reference; what it last moved by, as a power and a factor
  __shared__ float s_max[4 * W][NC], s_red[4 * W][NC], s_fin[2][N];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int Hp = P.H_kv * P.RG;
  const int range = blockIdx.x / Hp, gp = blockIdx.x % Hp;
  const int g = gp / P.RG, row0 = (gp % P.RG) * P.Rg;
  const int rows = min(P.Rg, P.R - row0);       // live rows of this CTA
  const int live0 = kl_first(rows, W);          // of a softmax warpgroup, but the last
  const int softmax_warps = 4 * ((rows + live0 - 1) / live0);
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t q_smem = smem_u32(smem);
  const uint32_t k_ring = q_smem + 2 * Cfg::kQ, v_ring = k_ring + KS * kTile;
  const uint32_t p_smem = v_ring + VS * kTile;

  // Lengths and block numbers are the caller's: the ranges and the first block
  // numbers are worked out while the kernel before this one runs.
  if (warp == 0) {
    bool bad;
    int4 split;
    const int64_t all = kl_all_tiles(P, bad);
    const int4 w = kl_range(P, range, all, split);
    if (lane == 0) s_work = w;
  } else if (tid == 32) {
    for (int k = 0; k < kChunks; ++k) {
      mbar_init(&page_full[k], 1);
      mbar_init(&scale_full[k], 1);
      mbar_init(&page_empty[k], 5 + softmax_warps);   // the K, V, MMA and scale warps, and those that read the scales
    }
    for (int k = 0; k < KS; ++k) {
      mbar_init(&k_full[k], 1);
      mbar_init(&k_empty[k], 1);
    }
    for (int k = 0; k < VS; ++k) {
      mbar_init(&v_full[k], 1);
      mbar_init(&v_empty[k], 1);
    }
    for (int k = 0; k < 2; ++k) {
      mbar_init(&drain[k], 1);
      mbar_init(&q_full[k], 1);
      mbar_init(&q_empty[k], 1);
      mbar_init(&o_free[k], softmax_warps);
      mbar_init(&s_full[k], 2);   // Q K^T of the step, and P V of the step before the last
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

  // Waits for the chunk that tile u opens; after a chunk's last tile a warp hands
  // it back.
  auto pages_wait = [&](uint32_t u, bool &ok) {
    if (u % kChunk == 0) ok = kl_wait(&page_full[u / kChunk % kChunks], (u / (kChunk * kChunks)) & 1, abf, P.wait_ns) && ok;
  };
  auto pages_done = [&](uint32_t u) {
    if (u % kChunk == kChunk - 1) {
      __syncwarp();
      if (lane == 0) mbar_arrive(&page_empty[u / kChunk % kChunks]);
    }
  };

  if (warp >= kPageWarp) regs_dec<Cfg::kRegsOther>();
  if (warp != kPageWarp) pdl_wait();
  pdl_trigger();
  if (warp == kPageWarp) {
    // ------------------------------------------------------- block numbers --
    KlWalk wk = kl_walk(P, work);
    KlItem it;
    bool have = kl_next(P, wk, it);
    int ti = 0;   // next tile of the item
    bool bad = false;
    for (int c = 0; c * kChunk < total; ++c) {
      if (c == kChunks) pdl_wait();   // (from here on it waits for warps that wait there)
      if (c >= kChunks &&
          !__all_sync(0xffffffffu, kl_wait(&page_empty[c % kChunks], ((c / kChunks) & 1) ^ 1, abf, P.wait_ns)))
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
          s_phys[(c % kChunks * kChunk + filled) * kTP + e] = ph;
        }
        if (lane < n) {
          const int tt = ti + lane, at = c % kChunks * kChunk + filled + lane;
          const int key0 = (it.tile0 + tt) * kTK, nv = min(kTP, it.span.nblk - (it.tile0 + tt) * kTP);
          int z0 = 0, z1 = 0;
          const bool edge = key0 + kTK - 1 > it.span.L - P.n_new || (P.window > 0 && key0 < it.span.L - P.window);
          if (P.window > 0) {   // between the sinks and the oldest query's window
            z0 = min(max(P.sinks - key0, 0), kTK);
            z1 = min(max(it.span.L - P.n_new - P.window + 1 - key0, 0), kTK);
            if (z0 >= z1) z0 = z1 = 0;
          }
          s_flag[at] = (tt == 0 ? kFirst : 0) | (tt == it.ntiles - 1 ? kLast | kEnd : 0) | (tt % T == T - 1 ? kEnd : 0) |
                       (tt % T ? kSecond : 0) | (edge ? kEdge : 0) | nv << 8;
          s_zero[at] = z0 | z1 << 8 | min(it.span.L - key0, kTK) << 16;
        }
        filled += n;
        ti += n;
        if (ti == it.ntiles) {
          have = kl_next(P, wk, it);
          ti = 0;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&page_full[c % kChunks]);
    }
    pdl_wait();
    if (bad) atomic_or_status(P.status, SV_DEV_BAD_BLOCK);
  } else if (warp == kScaleWarp) {
    // -------------------------------------------------------------- scales --
    const int64_t scales_at = q8_scale_offset(P.H_kv, kD, kBS) + 4 * g;
    bool ok = true;
    for (int c = 0; c * kChunk < total; ++c) {
      pages_wait(c * kChunk, ok);
      if (!__all_sync(0xffffffffu, ok)) break;
      constexpr int kE = kChunk * kTP / 32;
      const int n = min(kChunk, total - c * kChunk) * kTP, at = c % kChunks * kChunk * kTP;
      float ks[kE], vs[kE];
#pragma unroll
      for (int k = 0; k < kE; ++k) {
        ks[k] = vs[k] = 0.f;
        if (lane + 32 * k < n) {
          const int64_t off = (int64_t)s_phys[at + lane + 32 * k] * P.block_stride + scales_at;
          ks[k] = *reinterpret_cast<const float *>(P.k_cache + off);
          vs[k] = *reinterpret_cast<const float *>(P.v_cache + off);
        }
      }
#pragma unroll
      for (int k = 0; k < kE; ++k) {
        const float v = q8_scale(vs[k]);
        if (lane + 32 * k < n)
          s_scale[at + lane + 32 * k] = make_float4(q8_scale(ks[k]), lg2f(v), rcpf(v), s_flag[(at + lane + 32 * k) / kTP] & kEdge ? 1.f : 0.f);
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&scale_full[c % kChunks]);
        if ((c + 1) * kChunk <= total) mbar_arrive(&page_empty[c % kChunks]);
      }
    }
  } else if (warp == kKWarp || warp == kVWarp) {
    // ------------------------------------------------------ codes to smem --
    auto role = [&](auto is_v) {
      constexpr bool V = decltype(is_v)::value;
      constexpr int S = V ? VS : KS;
      uint64_t *full = V ? v_full : k_full, *empty = V ? v_empty : k_empty;
      const uint32_t ring = V ? v_ring : k_ring;
      const CUtensorMap *map = V ? &M.v : &M.k;
      bool ok = true;
      int u = 0, s = 0;
      uint32_t phase = 1;   // of `empty`, from the second round of the ring on
      const bool run = !(P.withhold & SV_TEST_WITHHOLD_COPIES);
      for (; run && u < total; ++u) {
        pages_wait(u, ok);
        if (u >= S) ok = kl_wait(&empty[s], phase, abf, P.wait_ns) && ok;
        if (!__all_sync(0xffffffffu, ok)) break;
        const int at = u % (kChunk * kChunks), nv = s_flag[at] >> 8;
        if (lane == 0) mbar_arrive_expect_tx(&full[s], nv * kBS * kD);
        __syncwarp();
        if (lane < nv) tma_load_4d(ring + s * kTile + lane * (kBS * kD), map, 0, 0, g, s_phys[at * kTP + lane], &full[s]);
        pages_done(u);
        if (++s == S) {
          s = 0;
          phase ^= 1;
        }
      }
      // the copies in flight land before the CTA may exit
      if (lane == 0)
        for (int k = max(0, u - S); k < u; ++k)
          if (!mbar_wait(&full[k % S], (k / S) & 1)) atomic_or_status(P.status, SV_DEV_TIMEOUT);
    };
    if (warp == kVWarp) role(std::true_type{});
    else role(std::false_type{});
  } else if (warp == kQWarp) {
    // ------------------------------------------------------------------- Q --
    KlWalk wk = kl_walk(P, work);
    KlItem it;
    int i = 0;
    while (kl_next(P, wk, it)) {
      const int buf = i & 1, row = i % 3;
      // the buffer after Q K^T of the item before the last, the rows after the
      // epilogue of the one before that
      bool ok = i < 2 || kl_wait(&q_empty[buf], ((i >> 1) & 1) ^ 1, abf, P.wait_ns);
      if (i >= 3) ok = kl_wait(&o_free[buf ^ 1], ((i - 3) >> 1) & 1, abf, P.wait_ns) && ok;
      if (!__all_sync(0xffffffffu, ok)) break;
      const int64_t ent = (int64_t)it.b * Hp + gp;
      const float *qs = P.ws_qs + ent * (2 * N + 4);
      const float fold = qs[N];
      for (int col = lane; col < N; col += 32) {
        const int w = col / CP, c = col - w * CP;
        const int r = row0 + (c < min(rows - w * live0, live0) ? w * live0 + c : 0);   // (padding: any)
        const int j = r / P.G;
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
    // One warp per product; all its lanes wait, one issues. f32 accumulators, M =
    // 128; Q K^T of e4m3 codes and terms, P V of e4m3 codes and e5m2 terms, both
    // read across their rows.
    constexpr uint32_t idesc_qk = (1u << 4) | ((uint32_t)(Cfg::kSCols >> 3) << 17) | (8u << 24);
    constexpr uint32_t idesc_pv = (1u << 4) | (1u << 10) | (1u << 15) | (1u << 16) | ((uint32_t)(Cfg::kOCols >> 3) << 17) | (8u << 24);
    uint32_t items = 0, step = 0;   // items started, steps done
    bool ok = true;
    uint32_t s = 0, round = 0;      // stage, and rounds of the ring
    if (warp == kQkWarp) {
      for (uint32_t u = 0; u < (uint32_t)total; ++u) {
        const uint32_t pb = step & 1;
        pages_wait(u, ok);
        const int flag = s_flag[u % (kChunks * kChunk)];
        if (flag & kFirst) {
          ok = kl_wait(&q_full[items & 1], (items >> 1) & 1, abf, P.wait_ns) && ok;
          ++items;
        }
        // the softmax of the step before the last has read the S buffers
        // (before there is one, the phase that counts as done)
        if (!(flag & kSecond)) ok = kl_wait2(&k_full[s], round & 1, &p_full[pb], ((step >> 1) & 1) ^ 1, abf, P.wait_ns) && ok;
        else ok = kl_wait(&k_full[s], round & 1, abf, P.wait_ns) && ok;
        if (!__all_sync(0xffffffffu, ok)) break;
        t5_fence_after();
        if (elect_one()) {
          const uint64_t qd = t5_desc(q_smem + ((items - 1) & 1) * Cfg::kQ, 16, 1024);
          const uint64_t kd = t5_desc(k_ring + s * kTile, 16, 1024);
          const uint32_t d = tb + Cfg::kSCol + (T * pb + (flag & kSecond ? 1 : 0)) * Cfg::kSCols;
#pragma unroll
          for (int kk = 0; kk < 8 / Cfg::kSSums; ++kk)   // 32 head dims per MMA, the hi terms of Q and the lo terms
            t5_mma_ss_f8(d, kd + (kk & 3) * 2, qd + (kk >> 2) * (N * 128 / 16) + (kk & 3) * 2, idesc_qk, kk > 0 ? 1u : 0u);
          t5_commit(&k_empty[s]);
          if (flag & kEnd) {
            t5_commit(&s_full[pb]);
          }
          if (flag & kLast) t5_commit(&q_empty[(items - 1) & 1]);
        }
        __syncwarp();
        pages_done(u);
        if (flag & kEnd) ++step;
        if (++s == KS) {
          s = 0;
          ++round;
        }
      }
    } else {
      if (lane < 2) mbar_arrive(&s_full[lane]);   // (no P V before the first steps)
      for (uint32_t u = 0; u < (uint32_t)total; ++u) {
        const uint32_t pb = step & 1;
        pages_wait(u, ok);
        const int at = u % (kChunks * kChunk), flag = s_flag[at], zero = s_zero[at];
        pages_done(u);
        if (flag & kFirst) {
          // O of the item before the last has been read
          if (items >= 2) ok = kl_wait(&o_free[items & 1], ((items >> 1) & 1) ^ 1, abf, P.wait_ns) && ok;
          ++items;
        }
        const int parts = ((flag >> 8) + 1) >> 1;   // of 32 keys that hold any
        const int z0 = zero & 255, z1 = (zero >> 8) & 255, z2 = zero >> 16;
        if (z1 > 0 || z2 < kTK) {
          // rows that no query sees become zeros: whatever they hold (NaN codes, or what an
          // earlier tile left), 0 times it would not do
          ok = __all_sync(0xffffffffu, kl_wait(&v_full[s], round & 1, abf, P.wait_ns)) && ok;
          const int n1 = (z1 - z0) * 8, n2 = (parts * 32 - z2) * 8;
          for (int i = lane; ok && i < n1 + n2; i += 32)
            asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(v_ring + s * kTile + (i < n1 ? z0 * kD + i * 16 : z2 * kD + (i - n1) * 16)),
                         "r"(0u)
                         : "memory");
          fence_proxy_async_shared();
          __syncwarp();
        }
        if (!(flag & kSecond)) ok = kl_wait2(&v_full[s], round & 1, &p_full[pb], (step >> 1) & 1, abf, P.wait_ns) && ok;
        else ok = kl_wait(&v_full[s], round & 1, abf, P.wait_ns) && ok;
        if (!__all_sync(0xffffffffu, ok)) break;
        t5_fence_after();
        if (elect_one()) {
          const uint64_t pd = t5_desc32(p_smem + (T * pb + (flag & kSecond ? 1 : 0)) * Cfg::kPBytes, Cfg::kAtom, 256);
          const uint64_t vd = t5_desc(v_ring + s * kTile, 16, 1024);
          const uint32_t d = tb + Cfg::kOCol + ((items - 1) & 1) * Cfg::kOCols;
          const uint32_t acc = flag & kFirst ? 0u : 1u;
          auto part = [&](int kk) {   // 32 keys
            t5_mma_ss_f8(d, vd + kk * (32 * kD / 16), pd + kk * (32 * 32 / 16), idesc_pv, kk > 0 ? 1u : acc);
          };
          if (parts == kTP / 2) {
#pragma unroll
            for (int kk = 0; kk < kTP / 2; ++kk) part(kk);
          } else {
#pragma unroll 1
            for (int kk = 0; kk < parts; ++kk) part(kk);
          }
          t5_commit(&v_empty[s]);
          if (flag & kEnd) {
            t5_commit(&pv_done[pb]);
            t5_commit(&s_full[pb]);   // the P' buffers are free: part of what the softmax of the step after next waits for
          }
        }
        __syncwarp();
        if (flag & kEnd) ++step;
        if (++s == VS) {
          s = 0;
          ++round;
        }
      }
    }
    // every MMA issued has completed before TMEM can be released
    if (total > 0) {
      uint64_t *dr = &drain[warp - kQkWarp];
      if (elect_one()) t5_commit(dr);
      __syncwarp();
      if (!mbar_wait(dr, 0) && lane == 0) atomic_or_status(P.status, SV_DEV_TIMEOUT);
    }
  } else if (warp < softmax_warps) {
    // ------------------------------------------------------------- softmax --
    regs_inc<Cfg::kRegsSoftmax>();
    const int w = warp >> 2, t = tid & 127;
    const int c_first = w * CP;                 // this warpgroup's columns
    const int live = min(rows - w * live0, live0);
    const int bar = 1 + w;
    const uint32_t lanes = tb + ((uint32_t)((warp & 3) * 32) << 16);
    // where this warpgroup's columns of each term begin in this key's row of P' (its two 16-byte
    // pieces are exchanged in every other four rows)
    uint32_t p_row[3];
#pragma unroll
    for (int e = 0; e < 3; ++e) {
      const uint32_t col = e * N + c_first;
      p_row[e] = p_smem + t * 32 + (col >> 5) * Cfg::kAtom + ((col & 24) ^ ((t << 2) & 16));
      if constexpr (W < 6) asm volatile("" : "+r"(p_row[e]));   // (kept, not worked out for every store, where registers allow)
    }
    int u = 0, i = 0;            // tiles and items done
    uint32_t step = 0;
    // A wait that gave up (ok false) only shows at the warpgroup's next vote, so
    // that its four warps leave together.
    bool ok = true;
    // The epilogue's second part, a head dim per thread: O of an item, once its
    // last P V is done; it is taken after the next item's first step, which hides
    // that P V.
    bool pending = false;   // (of item i - 1, whose last step was step - 1)
    auto finish = [&] {
      pending = false;
      const int buf = (i - 1) & 1, row = (i - 1) % 3, kind = s_item[row].w;
      const int64_t ent = 2 * (int64_t)blockIdx.x + (kind & kOpening ? 0 : 1);
      ok = __all_sync(0xffffffffu, kl_wait(&pv_done[(step - 1) & 1], ((step - 1) >> 1) & 1, abf, P.wait_ns)) && ok;
      if (!ok) return;
      t5_fence_after();
      float o[NC], o1[NC], o2[NC];
      const uint32_t at = lanes + Cfg::kOCol + buf * Cfg::kOCols + c_first;
      t5_ldn(at, reinterpret_cast<uint32_t(&)[NC]>(o));
      t5_ldn(at + N, reinterpret_cast<uint32_t(&)[NC]>(o1));
      t5_ldn(at + 2 * N, reinterpret_cast<uint32_t(&)[NC]>(o2));
      t5_wait_ld();
      keep_after<NC>(o);
      keep_after<NC>(o1);
      keep_after<NC>(o2);
#pragma unroll
      for (int k = 0; k < NC; ++k) {
        if (k >= live) break;
        const float x = fmaf(o2[k], kCut, o[k] + o1[k]) * s_fin[buf][c_first + k];
        if (kind & kWhole)
          static_cast<__nv_bfloat16 *>(P.out)[(int64_t)s_row[row][c_first + k] * kD + t] = __float2bfloat16_rn(x);
        else
          P.ws_acc[(ent * P.Rg + w * live0 + k) * kD + t] = x;
      }
      t5_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_free[buf]);
    };
    while (u < s_work.z) {
      const int buf = i % 3;
      const uint32_t o_col = lanes + Cfg::kOCol + (i & 1) * Cfg::kOCols + c_first;
      ok = __all_sync(0xffffffffu, kl_wait(&q_full[i & 1], (i >> 1) & 1, abf, P.wait_ns)) && ok;
      const float fold = P.scale_log2 * s_fold[buf];
      const int ntiles = s_item[buf].y;
      if (t < NC) s_nb[c_first + t] = t < live ? 0.f : -kUnset;   // (padding has no weight)
      bool open = true, unset = t < live;   // rows that have met no key; this thread's row among them
      float2 l2[NC / 2];
#pragma unroll
      for (int k = 0; k < NC / 2; ++k) l2[k] = make_float2(0.f, 0.f);
      bool gone = bar_or(bar, 128, !ok);
      for (int ti = 0; ti < ntiles && !gone; ++step) {
        const int nt = min(ntiles - ti, T);
        // S of this step, and with it the P' buffers that P V two steps ago has read
        const int pb = step & 1;
        float ka[T], vc[T], vi[T];
        bool edge[T];
#pragma unroll
        for (int h = 0; h < T; ++h) {   // this thread's keys
          if (h < nt && (u + h) % kChunk == 0)
            ok = kl_wait(&scale_full[(u + h) / kChunk % kChunks], ((u + h) / (kChunk * kChunks)) & 1, abf, P.wait_ns) && ok;
          const float4 s = s_scale[(u + h) % (kChunk * kChunks) * kTP + (t >> 4)];   // (of an absent tile: any)
          ka[h] = s.x * fabsf(fold);
          vc[h] = s.y;
          vi[h] = s.z;
          edge[h] = s.w != 0.f;
        }
        ok = kl_wait(&s_full[pb], (step >> 1) & 1, abf, P.wait_ns) && ok;
        const uint32_t s_col = lanes + Cfg::kSCol + T * pb * Cfg::kSCols + c_first;
        ok = __all_sync(0xffffffffu, ok);
        if (fold < 0.f && ok) kl_scale_rows<NC, N>(s_col, nt * Cfg::kSSums, &s_qf[buf][c_first]);   // rows with powers of their own
        t5_fence_after();
        float2 y[T][NC / 2];   // log2 weights, minus the reference
        {
          uint32_t v[T][Cfg::kSSums][NC];
          auto load = [&](int h) {
#pragma unroll
            for (int e = 0; e < Cfg::kSSums; ++e) t5_ldn(s_col + h * Cfg::kSCols + e * N, v[h][e]);
          };
          load(0);
          if (T > 1 && nt > 1) load(T - 1);
          float2 nb[NC / 2];
#pragma unroll
          for (int k = 0; k < NC; k += 4) {
            const float4 b = *reinterpret_cast<const float4 *>(&s_nb[c_first + k]);
            nb[k / 2] = make_float2(b.x, b.y);
            nb[k / 2 + 1] = make_float2(b.z, b.w);
          }
          t5_wait_ld();
          auto scores = [&](int h) {
#pragma unroll
            for (int e = 0; e < Cfg::kSSums; ++e) keep_after<NC>(reinterpret_cast<float(&)[NC]>(v[h][e]));
            const float2 ka2 = make_float2(ka[h], ka[h]), vc2 = make_float2(vc[h], vc[h]);
#pragma unroll
            for (int k = 0; k < NC / 2; ++k) {
              float2 q = make_float2(__uint_as_float(v[h][0][2 * k]), __uint_as_float(v[h][0][2 * k + 1]));
              if constexpr (Cfg::kSSums > 1) q = __fadd2_rn(q, make_float2(__uint_as_float(v[h][1][2 * k]), __uint_as_float(v[h][1][2 * k + 1])));
              y[h][k] = __ffma2_rn(q, ka2, __fadd2_rn(vc2, nb[k]));
            }
          };
          scores(0);
          if constexpr (T > 1) {
            if (nt > 1) {
              scores(T - 1);
            } else {
#pragma unroll
              for (int k = 0; k < NC / 2; ++k) y[T - 1][k] = make_float2(-INFINITY, -INFINITY);
            }
          }
        }
        // A tile that ends past the oldest query or holds keys that a window has
        // left: position j sees a key iff 0 <= j - j0 < reach.
#pragma unroll
        for (int h = 0; h < T; ++h)
          if (edge[h]) {
            const int4 at = s_item[buf];
            const int key = (at.x + ti + h) * kTK + t, j0 = key - (at.z - P.n_new);
            const uint32_t reach = P.window > 0 && key >= P.sinks ? (uint32_t)P.window : 0x80000000u;
#pragma unroll
            for (int k = 0; k < NC; k += 4) {
              const int4 j = *reinterpret_cast<const int4 *>(&s_pos[buf][c_first + k]);
              if ((uint32_t)(j.x - j0) >= reach) y[h][k / 2].x = -INFINITY;
              if ((uint32_t)(j.y - j0) >= reach) y[h][k / 2].y = -INFINITY;
              if ((uint32_t)(j.z - j0) >= reach) y[h][k / 2 + 1].x = -INFINITY;
              if ((uint32_t)(j.w - j0) >= reach) y[h][k / 2 + 1].y = -INFINITY;
            }
          }
        // Steps set the references of rows that have met no key yet (they are 0 so
        // far), and move those of rows with a weight above 2^kMove. All four warps
        // decide together, as they share O.
        float top = fmaxf(y[0][0].x, y[0][0].y);
#pragma unroll
        for (int k = 1; k < NC / 2; ++k) top = fmaxf(fmaxf(top, y[0][k].x), y[0][k].y);
        if constexpr (T > 1) {
#pragma unroll
          for (int k = 0; k < NC / 2; ++k) top = fmaxf(fmaxf(top, y[1][k].x), y[1][k].y);
        }
        bool moved = false;
        if (bar_or(bar, 128, open || top > kMove || !ok)) {
          if (bar_or(bar, 128, !ok)) {
            gone = true;
            break;
          }
          {   // each column's largest weight
            float v[NC];
#pragma unroll
            for (int k = 0; k < NC; ++k)
              v[k] = k & 1 ? fmaxf(y[0][k / 2].y, y[T - 1][k / 2].y) : fmaxf(y[0][k / 2].x, y[T - 1][k / 2].x);
            int at = 0, n = 0;
            warp_joined<NC, true>(v, lane, at, n);
#pragma unroll
            for (int k = 0; k < 5; ++k)   // (lanes with the same maxima write the same words)
              if (k < n) s_max[warp][at + k] = v[k];
          }
          named_bar_sync(bar, 128);
          if (t < NC) {
            float a = 1.f, by = 0.f;
            if (t < live) {
              const float m = fmaxf(fmaxf(s_max[4 * w][t], s_max[4 * w + 1][t]), fmaxf(s_max[4 * w + 2][t], s_max[4 * w + 3][t]));
              if (m > (unset ? -INFINITY : kMove)) {
                by = kTop - m;
                a = unset ? 1.f : ex2f(by);
                s_nb[c_first + t] += by;
                unset = false;
              }
            }
            s_by[c_first + t] = by;
            s_a[c_first + t] = a;
          }
          open = bar_or(bar, 128, unset);
#pragma unroll
          for (int k = 0; k < NC; k += 4) {
            const float4 by = *reinterpret_cast<const float4 *>(&s_by[c_first + k]);
            const float4 a = *reinterpret_cast<const float4 *>(&s_a[c_first + k]);
#pragma unroll
            for (int h = 0; h < T; ++h) {
              y[h][k / 2] = __fadd2_rn(y[h][k / 2], make_float2(by.x, by.y));
              y[h][k / 2 + 1] = __fadd2_rn(y[h][k / 2 + 1], make_float2(by.z, by.w));
            }
            l2[k / 2] = __fmul2_rn(l2[k / 2], make_float2(a.x, a.y));
            l2[k / 2 + 1] = __fmul2_rn(l2[k / 2 + 1], make_float2(a.z, a.w));
          }
          moved = ti > 0;
        }
        auto weights = [&](int h) {
          const float2 vi2 = make_float2(vi[h], vi[h]);
          const uint32_t at = (T * pb + h) * Cfg::kPBytes;
          constexpr int kEights = (NC + 7) / 8;   // pieces of eight columns: 8 or 16 bytes
          static_assert(kEights <= 2);
          uint2 piece[kEights][3];
#pragma unroll
          for (int c = 0; c < kEights; ++c) {
            uint32_t ph[4], w0[3], w1[3] = {};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int e = 4 * c + k;
              ph[k] = 0;
              if (e >= NC / 2) continue;
              const float2 p = make_float2(ex2f(y[h][e].x), ex2f(y[h][e].y));
              l2[e] = __ffma2_rn(p, vi2, l2[e]);
              ph[k] = pack2<true>(p.x, p.y);
            }
            cut_weights(ph[0], ph[1], w0);
            if (NC - 8 * c >= 8) cut_weights(ph[2], ph[3], w1);   // (what the columns of padding hold does not matter)
#pragma unroll
            for (int e = 0; e < 3; ++e) piece[c][e] = make_uint2(w0[e], w1[e]);
          }
#pragma unroll
          for (int e = 0; e < 3; ++e) {
            if constexpr (kEights == 1)
              asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(p_row[e] + at), "r"(piece[0][e].x), "r"(piece[0][e].y) : "memory");
            else
              asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(p_row[e] + at), "r"(piece[0][e].x), "r"(piece[0][e].y),
                           "r"(piece[1][e].x), "r"(piece[1][e].y)
                           : "memory");
          }
        };
        weights(0);
        if (T > 1 && nt > 1) weights(T - 1);
        if (moved) {   // O too, once the previous P V has landed (its wait lies behind the weights)
          ok = __all_sync(0xffffffffu, kl_wait(&pv_done[pb ^ 1], ((step - 1) >> 1) & 1, abf, P.wait_ns)) && ok;
          t5_fence_after();
          float o[3][NC];
#pragma unroll
          for (int e = 0; e < 3; ++e) t5_ldn(o_col + e * N, reinterpret_cast<uint32_t(&)[NC]>(o[e]));
          t5_wait_ld();
#pragma unroll
          for (int e = 0; e < 3; ++e) {
            keep_after<NC>(o[e]);
#pragma unroll
            for (int k = 0; k < NC; k += 4) {
              const float4 a = *reinterpret_cast<const float4 *>(&s_a[c_first + k]);
              o[e][k] *= a.x;
              o[e][k + 1] *= a.y;
              o[e][k + 2] *= a.z;
              o[e][k + 3] *= a.w;
            }
            t5_stn(o_col + e * N, reinterpret_cast<const uint32_t(&)[NC]>(o[e]));
          }
          t5_wait_st();
        }
        fence_proxy_async_shared();
        t5_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[pb]);
        __syncwarp();   // (what follows takes whole warps)
        pages_done(u);
        if (nt > 1) pages_done(u + 1);
        ti += nt;
        u += nt;
        if (pending) finish();
      }
      if (gone) break;
      // ---- epilogue, first part: sums over the keys -------------------------
      {
        float v[NC];
#pragma unroll
        for (int k = 0; k < NC; ++k) v[k] = k & 1 ? l2[k / 2].y : l2[k / 2].x;
        int at = 0, n = 0;
        warp_joined<NC, false>(v, lane, at, n);
#pragma unroll
        for (int k = 0; k < 5; ++k)   // (lanes with the same sums write the same words)
          if (k < n) s_red[warp][at + k] = v[k];
      }
      named_bar_sync(bar, 128);
      const int kind = s_item[buf].w;
      const int64_t ent = 2 * (int64_t)blockIdx.x + (kind & kOpening ? 0 : 1);
      if (t < live) {
        float l = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) l += s_red[4 * w + k][t];
        // (a row of NaN stays NaN; l is 0 only for a row without keys, which a query that sees itself never is)
        s_fin[i & 1][c_first + t] = kind & kWhole ? 1.f / l : 1.f;
        if (!(kind & kWhole)) {
          const int64_t e = ent * P.Rg + w * live0 + t;
          P.ws_ml[2 * e] = unset ? -kUnset : -s_nb[c_first + t];
          P.ws_ml[2 * e + 1] = l;
        }
      }
      pending = true;
      ++i;
    }
    named_bar_sync(bar, 128);
    if (pending) finish();
  }
  __syncthreads();
  if (tid == 0 && *abf) atomic_or_status(P.status, SV_DEV_TIMEOUT);
  t5_fence_after();
  if (warp == kQkWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tb), "r"(512));
}

template <int NC, int W>
sv_status launch_q8(const KlParams &P, const Q8Maps &M, int C, cudaStream_t st) {
  static DeviceOnce once;
  const cudaError_t err = once_per_device(once, [] {
    return cudaFuncSetAttribute(attn_q8_kernel<NC, W>, cudaFuncAttributeMaxDynamicSharedMemorySize, Q8Cfg<NC, W>::kSmem);
  });
  if (err != cudaSuccess) return fail(SV_ERR_CUDA, "spec_verify_attn_q8: cudaFuncSetAttribute: %s", cudaGetErrorString(err));
  const int64_t prep = (P.NR + kPrepWarps - 1) / kPrepWarps + (int64_t)P.B * P.H_kv * P.RG;
  launch_k(kl_prep_kernel<NC, W, false>, dim3((unsigned)prep), dim3(32 * kPrepWarps), 0, st, 1, P);
  launch_k(attn_q8_kernel<NC, W>, dim3(C), dim3(32 * Q8Cfg<NC, W>::kWarps), Q8Cfg<NC, W>::kSmem, st, 1, P, M);
  return check_launch("spec_verify_attn_q8 launch");
}

// Softmax warpgroups: 8 rows each as far as threads go, then 16. A step is a chain
// of waits that more warpgroups with shorter columns overlap better, as long as the
// registers suffice. 64 sequences of 4750 keys, 8 kv heads, captured: 32 rows, four of
// 8 120 us, two of 16 128; 40 rows, five of 8 132, six 143; 48 rows, six of 8 142, four
// of 16 168.
int q8_groups(int rows) { return rows <= 16 ? 2 : rows <= 32 ? 4 : rows <= 40 ? 5 : rows <= 48 ? 6 : 4; }

// Query rows of a kv head on the tensor cores: 64 share a pass over the cache.
constexpr int64_t kMaxRows = 1 << 14;

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" size_t spec_verify_attn_q8_workspace_size(int B, int n_new, int H_q, int H_kv, int d_head,
                                                     int max_blocks_per_seq, int block_size, int window, int sinks) {
  size_t other = spec_verify_attn_window_workspace_size(B, n_new, H_q, H_kv, d_head, max_blocks_per_seq,
                                                        block_size, window, sinks);
  if (other == 0) return 0;
  // (queries in f32 run on the CUDA-core kernel whatever the shape, as far as it takes their rows:
  // its partials of 2^14 rows would be gigabytes that no call can use)
  if (!attn_cuda_core_fits((int64_t)n_new * (H_q / H_kv), d_head)) other = 0;
  if ((int64_t)window >= (int64_t)max_blocks_per_seq * block_size) window = sinks = 0;
  const KlPlan p = kl_plan(B, n_new, H_q, H_kv, d_head, max_blocks_per_seq, block_size, SV_BF16, window, sinks, kMaxRows);
  return p.tc ? std::max(other, kl_ws_bytes(p, B, H_kv, q8_groups(p.Rg))) : other;
}

extern "C" sv_status spec_verify_attn_q8(const void *q, sv_dtype q_dtype, const void *k_cache, const void *v_cache,
                                         const sv_kv_layout *layout, const int32_t *block_table,
                                         int max_blocks_per_seq, const int32_t *seq_lens, int B, int n_new, int H_q,
                                         int H_kv, int d_head, int block_size, int num_blocks, float softmax_scale,
                                         int window, int sinks, void *out, sv_dtype out_dtype, void *workspace,
                                         size_t workspace_bytes, int32_t *dev_status, sv_stream_t stream) {
  if (window < 0 || sinks < 0) return fail(SV_ERR_INVALID_ARG, "spec_verify_attn_q8: negative window or sinks");
  if (max_blocks_per_seq > 0 && block_size > 0 && !capacity_ok(max_blocks_per_seq, block_size))
    return fail(SV_ERR_UNSUPPORTED, "spec_verify_attn_q8: max_blocks_per_seq * block_size must be below 2^30");
  KlPlan p = {};
  const bool sizes_ok = B >= 0 && n_new >= 1 && H_q >= 1 && H_kv >= 1 && H_q % H_kv == 0 && num_blocks >= 1 &&
                        max_blocks_per_seq >= 1 && H_kv <= 65535 && block_size >= 1;
  int win = window, snk = sinks;
  if ((int64_t)win >= (int64_t)max_blocks_per_seq * block_size) win = snk = 0;   // reaches every key
  if (sizes_ok) p = kl_plan(B, n_new, H_q, H_kv, d_head, max_blocks_per_seq, block_size, q_dtype, win, snk, kMaxRows);
  if (!p.tc || q_dtype != out_dtype)
    return attn_cuda_core_q8(q, q_dtype, k_cache, v_cache, layout, block_table, max_blocks_per_seq, seq_lens, B, n_new,
                             H_q, H_kv, d_head, block_size, num_blocks, softmax_scale, window, sinks, out, out_dtype,
                             workspace, workspace_bytes, dev_status, stream);
  if (!q || !k_cache || !v_cache || !block_table || !seq_lens || !out)
    return fail(SV_ERR_INVALID_ARG, "spec_verify_attn_q8: null pointer argument");
  if (!(softmax_scale > 0.f) || !std::isfinite(softmax_scale))
    return fail(SV_ERR_INVALID_ARG, "spec_verify_attn_q8: softmax_scale must be finite and > 0");
  KlParams P;
  memset(&P, 0, sizeof(P));
  const sv_status rc = q8_check("spec_verify_attn_q8", k_cache, v_cache, layout, H_kv, d_head, block_size, &P.block_stride);
  if (rc != SV_OK) return rc;
  const int W = q8_groups(p.Rg);
  const size_t need = B > 0 ? kl_ws_bytes(p, B, H_kv, W) : 0;
  if (!workspace || workspace_bytes < need)
    return fail(SV_ERR_WORKSPACE, "spec_verify_attn_q8: workspace needs %zu bytes", need);
  if (!aligned(workspace, 256)) return fail(SV_ERR_WORKSPACE, "spec_verify_attn_q8: workspace not 256-byte aligned");
  if (!aligned(q, 16) || !aligned(out, 16))
    return fail(SV_ERR_INVALID_ARG, "spec_verify_attn_q8: q and out must be 16-byte aligned");
  if (B == 0) return ok();
  PFN_cuTensorMapEncodeTiled_v12000 enc = get_encode();
  if (!enc) return fail(SV_ERR_CUDA, "spec_verify_attn_q8: cuTensorMapEncodeTiled unavailable");
  Q8Maps M;
  const cuuint64_t dims[4] = {(cuuint64_t)kD, (cuuint64_t)kBS, (cuuint64_t)H_kv, (cuuint64_t)num_blocks};
  const cuuint64_t strides[3] = {(cuuint64_t)kD, (cuuint64_t)kD * kBS, (cuuint64_t)P.block_stride};
  const cuuint32_t box[4] = {(cuuint32_t)kD, (cuuint32_t)kBS, 1, 1}, ones[4] = {1, 1, 1, 1};
  for (int w = 0; w < 2; ++w) {
    const CUresult r = enc(w ? &M.v : &M.k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void *>(w ? v_cache : k_cache), dims,
                           strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(SV_ERR_INVALID_ARG, "spec_verify_attn_q8: cuTensorMapEncodeTiled failed (%d)", (int)r);
  }
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
  at += align_up((size_t)B * H_kv * p.RG * kl_cols(p, W) * 256, 256);
  P.ws_qs = reinterpret_cast<float *>(at);
  P.status = dev_status;
  P.B = B; P.n_new = n_new; P.H_q = H_q; P.H_kv = H_kv; P.G = H_q / H_kv; P.R = p.R; P.Rg = p.Rg; P.RG = p.RG;
  P.NR = p.NR; P.max_blocks = max_blocks_per_seq; P.num_blocks = num_blocks; P.window = win; P.sinks = snk;
  P.scale_log2 = (float)((double)softmax_scale * 1.4426950408889634074);
  P.wait_ns = wait_limit_ns();
  P.withhold = test_withhold();
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int each = kl_first(p.Rg, W);   // rows of a softmax warpgroup
  const sv_status r2 = W == 6     ? launch_q8<8, 6>(P, M, p.C, st)
                       : W == 5   ? launch_q8<8, 5>(P, M, p.C, st)
                       : W == 2   ? (each <= 4 ? launch_q8<4, 2>(P, M, p.C, st) : launch_q8<8, 2>(P, M, p.C, st))
                       : each <= 8 ? launch_q8<8, 4>(P, M, p.C, st)
                                   : launch_q8<16, 4>(P, M, p.C, st);
  if (r2 != SV_OK || p.NR == 1) return r2;
  launch_k(kl_merge_kernel, dim3((p.NR - 1) * H_kv * p.RG, (p.Rg + kMergeWarps - 1) / kMergeWarps),
           dim3(32 * kMergeWarps), 0, st, 1, P);
  return check_launch("spec_verify_attn_q8 merge launch");
}
