// kv_block_append_q8 and kv_block_gather_q8: the 8-bit block-scaled paged
// cache's write and read-back (page layout: q8.cuh).
//
// For the new rows x of one (block, kv head), with A their largest magnitude
// (NaN left out):
//   e = the smallest integer with A <= 448 * 2^e, kept within -32..32 (A = 0: -32)
//   scale = 2^e if the rows start at slot 0, else max(old scale, 2^e)
//   code = e4m3(x / scale), to nearest even, saturated at +-448; NaN becomes 0
// and where the scale of a block that holds rows grows, their codes are moved:
// e4m3(code * old / new).
#include <algorithm>
#include <cstring>

#include "q8.cuh"
#include "tc5.cuh"

namespace sv {
namespace {

struct Q8AppendArgs {
  const void *src[2];   // K, V rows [B][n_new][H_kv][d]
  uint8_t *cache[2];
  const int32_t *block_table, *seq_lens;
  int max_blocks, n_new, H_kv, d, bs, num_blocks, pages;   // pages: blocks that n_new rows can touch
  int64_t block_stride;   // bytes
  int32_t *status;
};

constexpr int kEaWarps = 8;
constexpr int kEaBatch = 4;   // pieces of 16 elements that a lane holds

// Sixteen consecutive elements of a row, aligned to `to` bytes (32, 16, or less).
template <typename T>
__device__ __forceinline__ void load16(const T *p, int to, T (&x)[16]) {
  uint32_t *w = reinterpret_cast<uint32_t *>(x);
  if (to == 32) {
#pragma unroll
    for (int k = 0; k < 4 * (int)sizeof(T); k += 8)
      asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                   : "=r"(w[k]), "=r"(w[k + 1]), "=r"(w[k + 2]), "=r"(w[k + 3]), "=r"(w[k + 4]), "=r"(w[k + 5]),
                     "=r"(w[k + 6]), "=r"(w[k + 7])
                   : "l"(reinterpret_cast<const uint32_t *>(p) + k));
  } else if (to == 16) {
#pragma unroll
    for (int k = 0; k < (int)sizeof(T); ++k) reinterpret_cast<uint4 *>(x)[k] = reinterpret_cast<const uint4 *>(p)[k];
  } else {
#pragma unroll
    for (int k = 0; k < 16; ++k) x[k] = p[k];
  }
}
template <typename T>
__device__ __forceinline__ void store16(T *p, int to, const T (&x)[16]) {
  const uint32_t *w = reinterpret_cast<const uint32_t *>(x);
  if (to == 32) {
#pragma unroll
    for (int k = 0; k < 4 * (int)sizeof(T); k += 8)
      asm volatile("st.global.v8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(w[k]), "r"(w[k + 1]), "r"(w[k + 2]),
                   "r"(w[k + 3]), "r"(w[k + 4]), "r"(w[k + 5]), "r"(w[k + 6]), "r"(w[k + 7]),
                   "l"(reinterpret_cast<uint32_t *>(p) + k)
                   : "memory");
  } else if (to == 16) {
#pragma unroll
    for (int k = 0; k < (int)sizeof(T); ++k) reinterpret_cast<uint4 *>(p)[k] = reinterpret_cast<const uint4 *>(x)[k];
  } else {
#pragma unroll
    for (int k = 0; k < 16; ++k) p[k] = x[k];
  }
}

__device__ __forceinline__ float fmax_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The largest magnitude of x and m; a NaN among them stays.
__device__ __forceinline__ float amax16(const __nv_bfloat16 (&x)[16], float m) {
  __nv_bfloat162 t = __habs2(reinterpret_cast<const __nv_bfloat162 *>(x)[0]);
#pragma unroll
  for (int k = 1; k < 8; ++k) t = __hmax2_nan(t, __habs2(reinterpret_cast<const __nv_bfloat162 *>(x)[k]));
  return fmax_nan(fmax_nan(__low2float(t), __high2float(t)), m);
}
__device__ __forceinline__ float amax16(const float (&x)[16], float m) {
#pragma unroll
  for (int k = 0; k < 16; ++k) m = fmax_nan(m, fabsf(x[k]));
  return m;
}

// NaN as 0.
template <typename T>
__device__ __forceinline__ void drop_nan(T (&x)[16]) {
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const float v = to_f32(x[k]);
    if (v != v) x[k] = T(0.f);
  }
}

// The smallest e with a <= 448 * 2^e (448 = 1.75 * 2^8), within +-32.
__device__ __forceinline__ int q8_exponent(float a) {
  const uint32_t bits = __float_as_uint(a);
  const int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, -kQ8MaxExp), kQ8MaxExp);
}

// Codes of sixteen elements: x by `by`, or (DIV) over it.
template <bool DIV, typename T>
__device__ __forceinline__ uint4 codes16(const T (&x)[16], float by) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float v = to_f32(x[4 * k + e]);
      y[e] = DIV ? __fdiv_rn(v, by) : v * by;
    }
    w[k] = f32x2_to_e4m3x2(y[0], y[1]) | (f32x2_to_e4m3x2(y[2], y[3]) << 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float2 e4m3x2_to_f32x2(uint32_t codes) {
  const uint32_t h = e4m3x2_to_f16x2((uint16_t)codes);
  return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// A warp takes the new rows of one (block written, kv head) of K or of V: largest
// magnitude and codes from one read, the rows in registers between.
// Bound by memory, with the instructions not far behind: 16 prompts of 2047 rows, 8
// kv heads of 128, 134 MB read and 67 MB written, take 36 us (52 with a division
// chosen per element; 16-byte reads, which fetch each sector twice, and NaN looked
// for per element cost another 10). The batch and the four CTAs an SM suit bf16: f32
// rows spill, the same rows take 85 us against 50 of their bytes.
template <typename T>
__global__ void __launch_bounds__(32 * kEaWarps, 4) q8_append_kernel(const __grid_constant__ Q8AppendArgs a, int to) {
  pdl_trigger();
  const int lane = threadIdx.x & 31, b = blockIdx.y;
  const unsigned unit = blockIdx.x * kEaWarps + (threadIdx.x >> 5);
  const int kv = (int)(unit & 1), g = (int)((unit >> 1) % (unsigned)a.H_kv);
  const int64_t p = (unit >> 1) / (unsigned)a.H_kv;
  const int bs = a.bs, d = a.d, L = a.seq_lens[b];
  const bool len_ok = L >= a.n_new && L <= a.max_blocks * bs;
  const int first = L - a.n_new;
  const int64_t page = first / bs + p;
  const int s0 = (int)max(first - page * bs, (int64_t)0), s1 = (int)min(L - page * bs, (int64_t)bs);   // slots written
  const bool mine = len_ok && p < a.pages && s0 < s1;
  const int phys = mine ? a.block_table[(int64_t)b * a.max_blocks + page] : 0;
  // the new rows may be what the kernel before writes (a rotation, a read-back),
  // and the pools may still be read by it
  pdl_wait();
  if (!len_ok && lane == 0 && unit == 0) atomic_or_status(a.status, SV_DEV_BAD_SEQ_LEN);
  if (!mine) return;
  const int C = d / 16, n = (s1 - s0) * C;   // pieces of 16 elements in a row, and in all
  const int64_t row_stride = (int64_t)a.H_kv * d;
  const T *src = static_cast<const T *>(a.src[kv]) + (((int64_t)b * a.n_new + (page * bs + s0 - first)) * a.H_kv + g) * d;
  alignas(16) T x[kEaBatch][16];
  auto fetch = [&](int i0) {
#pragma unroll
    for (int k = 0; k < kEaBatch; ++k) {
      const int i = i0 + 32 * k + lane;
      if (i < n) load16(src + (int64_t)(i / C) * row_stride + (i % C) * 16, to, x[k]);
    }
  };
  const bool once = n <= 32 * kEaBatch;   // the rows stay in registers
  fetch(0);
  if (phys < 0 || phys >= a.num_blocks) {
    if (lane == 0) atomic_or_status(a.status, SV_DEV_BAD_BLOCK);
    return;
  }
  uint8_t *pg = a.cache[kv] + (int64_t)phys * a.block_stride;
  uint8_t *codes = pg + (int64_t)g * bs * d;
  float *scale_at = reinterpret_cast<float *>(pg + q8_scale_offset(a.H_kv, d, bs)) + g;
  auto drop = [&] {
#pragma unroll
    for (int k = 0; k < kEaBatch; ++k) drop_nan(x[k]);
  };
  auto largest = [&](bool nan) {
    float top = 0.f;
    for (int i0 = 0; i0 < n; i0 += 32 * kEaBatch) {
      if (i0 > 0 || (nan && !once)) fetch(i0);
      if (nan) drop();
#pragma unroll
      for (int k = 0; k < kEaBatch; ++k)
        if (i0 + 32 * k + lane < n) top = amax16(x[k], top);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmax_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
    return top;
  };
  float top = largest(false);
  const bool nan = top != top;   // rare: once more without it
  if (nan) top = largest(true);
  const float fresh = __uint_as_float((uint32_t)(127 + q8_exponent(top)) << 23);
  float s = fresh;
  if (s0 > 0) {
    const float old = q8_scale(*scale_at);
    s = fmaxf(old, fresh);
    if (s > old) {   // the codes of the other slots move to the new scale
      const float ratio = old / s;
      for (int i = lane; i < bs * C; i += 32) {
        const int slot = i / C;
        if (slot >= s0 && slot < s1) continue;
        uint4 *at = reinterpret_cast<uint4 *>(codes) + i;
        uint4 w = *at;
        uint32_t *v = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 lo = e4m3x2_to_f32x2(v[k] & 0xffffu), hi = e4m3x2_to_f32x2(v[k] >> 16);
          v[k] = f32x2_to_e4m3x2(lo.x * ratio, lo.y * ratio) | (f32x2_to_e4m3x2(hi.x * ratio, hi.y * ratio) << 16);
        }
        *at = w;
      }
    }
    __syncwarp();   // every lane has read the old scale
  }
  if (lane == 0) *scale_at = s;
  // (a page written elsewhere may hold a scale that is no power of two)
  const uint32_t bits = __float_as_uint(s);
  const float inv = (bits & 0x7fffffu) == 0 ? __uint_as_float((254u << 23) - bits) : 0.f;
  for (int i0 = 0; i0 < n; i0 += 32 * kEaBatch) {
    if (!once) {
      fetch(i0);
      if (nan) drop();
    }
#pragma unroll
    for (int k = 0; k < kEaBatch; ++k) {
      const int i = i0 + 32 * k + lane;
      if (i >= n) continue;
      uint4 *at = reinterpret_cast<uint4 *>(codes) + s0 * C + i;
      if (inv != 0.f) *at = codes16<false>(x[k], inv);
      else *at = codes16<true>(x[k], s);
    }
  }
}

struct Q8GatherArgs {
  const uint8_t *cache[2];
  void *out[2];   // [B][n_rows][H_kv][d]
  const int32_t *block_table, *seq_lens, *start;
  int max_blocks, n_rows, H_kv, d, bs, num_blocks, pages;   // pages: blocks that n_rows rows can touch
  int64_t block_stride;   // bytes
  int32_t *status;
};

// Sixteen codes times s to sixteen consecutive elements of a row.
template <typename T>
__device__ __forceinline__ void write16(T *dst, int to, uint4 codes, float s) {
  const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
  alignas(16) T v[16];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float2 f = e4m3x2_to_f32x2((w[k / 2] >> (16 * (k & 1))) & 0xffffu);
    if constexpr (sizeof(T) == 4) {
      v[2 * k] = f.x * s;
      v[2 * k + 1] = f.y * s;
    } else {
      reinterpret_cast<__nv_bfloat162 *>(v)[k] = __floats2bfloat162_rn(f.x * s, f.y * s);
    }
  }
  store16(dst, to, v);
}

// A warp takes one block of one kv head, of K or of V. Rows outside the
// sequence, and those of a block with a number out of range, are written as
// zeros.
// Bound by memory: 16 prefixes of 4096 .. 8192 rows, 8 kv heads of 128, 739 MB read
// and written, take 114 us (144 with 16-byte stores, which write each sector in two
// pieces; two blocks a warp 116, four 118).
constexpr int kEgWarps = 8;
constexpr int kEgBatch = 4;   // pieces of 16 codes that a lane holds
template <typename T>
__global__ void __launch_bounds__(32 * kEgWarps, 5) q8_gather_kernel(const __grid_constant__ Q8GatherArgs a, int to) {
  pdl_trigger();
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  const unsigned unit = blockIdx.x * kEgWarps + (threadIdx.x >> 5);
  const int kv = (int)(unit & 1), g = (int)((unit >> 1) % (unsigned)a.H_kv);
  const int p = (int)((unit >> 1) / (unsigned)a.H_kv);
  const int bs = a.bs, d = a.d;
  const int L = a.seq_lens[b], start = a.start[b];
  const bool len_ok = L >= 0 && L <= a.max_blocks * bs;
  const int64_t page = (start >= 0 ? start / bs : -((bs - 1 - (int64_t)start) / bs)) + p;
  const int64_t i0 = page * bs - start;   // output row of slot 0
  const int r0 = (int)max((int64_t)0, -i0), r1 = (int)min((int64_t)bs, a.n_rows - i0);   // slots to write
  const bool mine = p < a.pages && r0 < r1;
  int held = mine && len_ok && page >= 0 ? (int)min((int64_t)bs, max((int64_t)0, L - page * bs)) : 0;   // slots that hold rows
  int phys = held > 0 ? a.block_table[(int64_t)b * a.max_blocks + page] : 0;
  pdl_wait();
  if (!len_ok && lane == 0 && unit == 0) atomic_or_status(a.status, SV_DEV_BAD_SEQ_LEN);
  if (!mine) return;
  if (phys < 0 || phys >= a.num_blocks) {
    if (lane == 0) atomic_or_status(a.status, SV_DEV_BAD_BLOCK);
    phys = held = 0;
  }
  const uint8_t *pg = a.cache[kv] + (int64_t)phys * a.block_stride;
  const uint4 *codes = reinterpret_cast<const uint4 *>(pg + (int64_t)g * bs * d);
  const int C = d / 16;
  const int64_t stride = (int64_t)a.H_kv * d;
  T *out = static_cast<T *>(a.out[kv]) + ((int64_t)b * a.n_rows + i0) * stride + (int64_t)g * d;   // of slot 0
  const float s = held > 0 ? q8_scale(reinterpret_cast<const float *>(pg + q8_scale_offset(a.H_kv, d, bs))[g]) : 0.f;
  for (int k0 = r0 * C; k0 < r1 * C; k0 += 32 * kEgBatch) {
    uint4 w[kEgBatch];
#pragma unroll
    for (int k = 0; k < kEgBatch; ++k) {
      const int i = k0 + 32 * k + lane;
      w[k] = make_uint4(0u, 0u, 0u, 0u);
      if (i < min(r1, held) * C) w[k] = codes[i];
    }
#pragma unroll
    for (int k = 0; k < kEgBatch; ++k) {
      const int i = k0 + 32 * k + lane;
      if (i < r1 * C) write16(out + (i / C) * stride + (i % C) * 16, to, w[k], s);
    }
  }
}

}  // namespace

// What the 8-bit entry points share: sizes, alignment and the page stride.
sv_status q8_check(const char *what, const void *k_cache, const void *v_cache, const sv_kv_layout *layout, int H_kv,
                   int d_head, int block_size, int64_t *block_stride) {
  if (d_head % 16 || d_head > 256 || block_size > 64)
    return fail(SV_ERR_UNSUPPORTED, "%s: 8-bit pools take d_head a multiple of 16 up to 256 and block_size up to 64", what);
  const int64_t page = q8_page_bytes(H_kv, d_head, block_size);
  *block_stride = layout ? layout->block_stride : page;
  if (*block_stride < page || *block_stride % 16 || (layout && (layout->head_stride != 0 || layout->slot_stride != 0)))
    return fail(SV_ERR_INVALID_ARG,
                "%s: the layout of an 8-bit pool has a page stride in bytes (a multiple of 16, at least %lld), "
                "head_stride 0 and slot_stride 0",
                what, (long long)page);
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16))
    return fail(SV_ERR_INVALID_ARG, "%s: 8-bit pools must be 16-byte aligned", what);
  return SV_OK;
}

}  // namespace sv

extern "C" size_t sv_q8_page_bytes(int H_kv, int d_head, int block_size) {
  if (H_kv < 1 || H_kv > 65535 || d_head < 16 || d_head % 16 || d_head > 256 || block_size < 1 || block_size > 64) return 0;
  return (size_t)sv::q8_page_bytes(H_kv, d_head, block_size);
}

extern "C" sv_status kv_block_append_q8(const void *k_new, const void *v_new, sv_dtype new_dtype, void *k_cache,
                                        void *v_cache, const sv_kv_layout *layout, const int32_t *block_table,
                                        int max_blocks_per_seq, const int32_t *seq_lens, int B, int n_new, int H_kv,
                                        int d_head, int block_size, int num_blocks, int32_t *dev_status,
                                        sv_stream_t stream) {
  using namespace sv;
  if (!k_new || !v_new || !k_cache || !v_cache || !block_table || !seq_lens)
    return fail(SV_ERR_INVALID_ARG, "kv_block_append_q8: null pointer argument");
  if (B < 0 || n_new < 1 || H_kv < 1 || d_head < 1 || block_size < 1 || num_blocks < 1 || max_blocks_per_seq < 1)
    return fail(SV_ERR_INVALID_ARG, "kv_block_append_q8: bad sizes");
  if (new_dtype != SV_F32 && new_dtype != SV_BF16)
    return fail(SV_ERR_UNSUPPORTED, "kv_block_append_q8: new rows must be f32 or bf16");
  if (B > 65535 || H_kv > 65535) return fail(SV_ERR_UNSUPPORTED, "kv_block_append_q8: B or H_kv too large");
  if (!capacity_ok(max_blocks_per_seq, block_size))
    return fail(SV_ERR_UNSUPPORTED, "kv_block_append_q8: max_blocks_per_seq * block_size must be below 2^30");
  Q8AppendArgs a = {};
  const sv_status rc = q8_check("kv_block_append_q8", k_cache, v_cache, layout, H_kv, d_head, block_size, &a.block_stride);
  if (rc != SV_OK) return rc;
  if (B == 0) return ok();
  a.src[0] = k_new; a.src[1] = v_new;
  a.cache[0] = static_cast<uint8_t *>(k_cache); a.cache[1] = static_cast<uint8_t *>(v_cache);
  a.block_table = block_table; a.seq_lens = seq_lens; a.max_blocks = max_blocks_per_seq; a.n_new = n_new;
  a.H_kv = H_kv; a.d = d_head; a.bs = block_size; a.num_blocks = num_blocks; a.status = dev_status;
  a.pages = (int)std::min<int64_t>(((int64_t)n_new + block_size - 2) / block_size + 1, max_blocks_per_seq);
  const int64_t units = (int64_t)a.pages * H_kv * 2, ctas = (units + kEaWarps - 1) / kEaWarps;
  if (units >= (1ll << 31)) return fail(SV_ERR_UNSUPPORTED, "kv_block_append_q8: too many rows");
  const int to = aligned(k_new, 32) && aligned(v_new, 32) ? 32 : aligned(k_new, 16) && aligned(v_new, 16) ? 16 : 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const dim3 grid((unsigned)ctas, B), block(32 * kEaWarps);
  if (new_dtype == SV_F32) launch_k(q8_append_kernel<float>, grid, block, 0, s, 1, a, to);
  else launch_k(q8_append_kernel<__nv_bfloat16>, grid, block, 0, s, 1, a, to);
  return check_launch("kv_block_append_q8 launch");
}

extern "C" sv_status kv_block_gather_q8(const void *k_cache, const void *v_cache, const sv_kv_layout *layout,
                                        const int32_t *block_table, int max_blocks_per_seq, const int32_t *seq_lens,
                                        const int32_t *start, int B, int n_rows, int H_kv, int d_head, int block_size,
                                        int num_blocks, void *k_out, void *v_out, sv_dtype out_dtype,
                                        int32_t *dev_status, sv_stream_t stream) {
  using namespace sv;
  if (!k_cache || !v_cache || !block_table || !seq_lens || !start || !k_out || !v_out)
    return fail(SV_ERR_INVALID_ARG, "kv_block_gather_q8: null pointer argument");
  if (B < 0 || n_rows < 0 || H_kv < 1 || d_head < 1 || block_size < 1 || num_blocks < 1 || max_blocks_per_seq < 1)
    return fail(SV_ERR_INVALID_ARG, "kv_block_gather_q8: bad sizes");
  if (out_dtype != SV_F32 && out_dtype != SV_BF16)
    return fail(SV_ERR_UNSUPPORTED, "kv_block_gather_q8: rows are read back as f32 or bf16");
  if (B > 65535 || H_kv > 65535) return fail(SV_ERR_UNSUPPORTED, "kv_block_gather_q8: B or H_kv too large");
  if (!capacity_ok(max_blocks_per_seq, block_size))
    return fail(SV_ERR_UNSUPPORTED, "kv_block_gather_q8: max_blocks_per_seq * block_size must be below 2^30");
  Q8GatherArgs a = {};
  const sv_status rc = q8_check("kv_block_gather_q8", k_cache, v_cache, layout, H_kv, d_head, block_size, &a.block_stride);
  if (rc != SV_OK) return rc;
  if (B == 0 || n_rows == 0) return ok();
  a.cache[0] = static_cast<const uint8_t *>(k_cache); a.cache[1] = static_cast<const uint8_t *>(v_cache);
  a.out[0] = k_out; a.out[1] = v_out; a.block_table = block_table; a.seq_lens = seq_lens; a.start = start;
  a.max_blocks = max_blocks_per_seq; a.n_rows = n_rows; a.H_kv = H_kv; a.d = d_head; a.bs = block_size;
  a.num_blocks = num_blocks; a.status = dev_status;
  a.pages = (int)(((int64_t)n_rows + block_size - 2) / block_size + 1);
  const int64_t units = (int64_t)a.pages * H_kv * 2, ctas = (units + kEgWarps - 1) / kEgWarps;
  if (units >= (1ll << 31)) return fail(SV_ERR_UNSUPPORTED, "kv_block_gather_q8: too many rows");
  const int to = aligned(k_out, 32) && aligned(v_out, 32) ? 32 : aligned(k_out, 16) && aligned(v_out, 16) ? 16 : 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const dim3 grid((unsigned)ctas, B), block(32 * kEgWarps);
  if (out_dtype == SV_F32) launch_k(q8_gather_kernel<float>, grid, block, 0, s, 1, a, to);
  else launch_k(q8_gather_kernel<__nv_bfloat16>, grid, block, 0, s, 1, a, to);
  return check_launch("kv_block_gather_q8 launch");
}
