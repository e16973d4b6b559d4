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

constexpr int kQaWarps = 8;

// NE consecutive elements of a row as floats; `vec`: the address is a multiple
// of the group's size.
template <typename T, int NE>
__device__ __forceinline__ void load_row(const T *p, bool vec, float (&x)[NE]) {
  if constexpr (sizeof(T) * NE % 8 == 0) {
    if (vec) {
      constexpr int NW = sizeof(T) * NE / 8;
      uint2 w[NW];
#pragma unroll
      for (int k = 0; k < NW; ++k) w[k] = __ldg(reinterpret_cast<const uint2 *>(p) + k);
      const T *e = reinterpret_cast<const T *>(w);
#pragma unroll
      for (int k = 0; k < NE; ++k) x[k] = to_f32(e[k]);
      return;
    }
  }
#pragma unroll
  for (int k = 0; k < NE; ++k) x[k] = to_f32(__ldg(p + k));
}

// One CTA per (block that new rows land in, kv head, sequence). A warp takes a
// row, NE = d / 32 elements a lane: minimum, maximum and codes, which go to
// shared memory a byte each; the CTA then packs them, K along the head dim and
// V along the slots, four bytes (eight codes) a thread. Words of a V record
// that also hold codes of other slots are read and merged; no other CTA of the
// call touches the record.
template <typename TIn, int NE>
__global__ void __launch_bounds__(32 * kQaWarps) q4_append_kernel(const __grid_constant__ Q4AppendArgs a, bool vec) {
  constexpr int d = 32 * NE;
  extern __shared__ __align__(16) uint8_t qa_codes[];   // [2][bs][d]
  pdl_trigger();
  const int g = blockIdx.y, b = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int bs = a.bs;
  const int L = a.seq_lens[b];
  if (L < a.n_new || L > a.max_blocks * bs) {
    if (threadIdx.x == 0 && g == 0 && blockIdx.x == 0) atomic_or_status(a.status, SV_DEV_BAD_SEQ_LEN);
    return;
  }
  const int first = L - a.n_new;
  const int page = first / bs + (int)blockIdx.x;
  const int s0 = max(first - page * bs, 0), s1 = min(L - page * bs, bs);   // slots written
  if (s0 >= s1) return;
  const int phys = a.block_table[(int64_t)b * a.max_blocks + page];
  if (phys < 0 || phys >= a.num_blocks) {
    if (threadIdx.x == 0) atomic_or_status(a.status, SV_DEV_BAD_BLOCK);
    return;
  }
  const int64_t rec = (int64_t)phys * a.block_stride + (int64_t)g * a.head_stride;
  const int nr = s1 - s0;
  bool waited = false;
  for (int i = warp; i < 2 * nr; i += kQaWarps) {
    const int kv = i >= nr ? 1 : 0, slot = s0 + i - kv * nr;
    const int j = page * bs + slot - first;
    const TIn *src = static_cast<const TIn *>(a.src[kv]) + (((int64_t)b * a.n_new + j) * a.H_kv + g) * d + lane * NE;
    float x[NE];
    load_row<TIn, NE>(src, vec, x);
    float mn = x[0], mx = x[0];   // (fminf and fmaxf leave NaN out)
#pragma unroll
    for (int k = 1; k < NE; ++k) {
      mn = fminf(mn, x[k]);
      mx = fmaxf(mx, x[k]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    }
    if (!(mn <= mx)) mn = mx = 0.f;   // nothing but NaN
    const __half mh = __float2half_rn(fminf(fmaxf(mn, -65504.f), 65504.f));
    const float m = __half2float(mh);
    const __half sh = __hmax(__float2half_rn(fminf(__fdiv_rn(__fsub_rn(mx, m), 15.f), 65504.f)), __ushort_as_half(1));
    const float s = __half2float(sh);
    uint8_t *dst = qa_codes + (kv * bs + slot) * d + lane * NE;
#pragma unroll
    for (int k = 0; k < NE; ++k)
      dst[k] = (uint8_t)(int)fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(x[k], m), s)), 0.f), 15.f);
    // everything read so far is the caller's; the pools may still be read by
    // the previous kernel of the stream
    if (!waited) {
      pdl_wait();
      waited = true;
    }
    if (lane == 0) {
      const uint32_t pair = (uint32_t)__half_as_ushort(sh) | ((uint32_t)__half_as_ushort(mh) << 16);
      *reinterpret_cast<uint32_t *>(a.cache[kv] + rec + q4_code_bytes(d, bs) + 4 * slot) = pair;
    }
  }
  if (!waited) pdl_wait();
  __syncthreads();
  // K: eight head dims of a slot per word
  for (int i = threadIdx.x; i < nr * (d / 8); i += 32 * kQaWarps) {
    const int slot = s0 + i / (d / 8), c = 8 * (i % (d / 8));
    const uint8_t *p = qa_codes + slot * d + c;
    uint32_t w = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) w |= (uint32_t)p[k] << (4 * k);
    *reinterpret_cast<uint32_t *>(a.cache[0] + rec + q4_k_byte(slot, c, d)) = w;
  }
  // V: eight slots of a head dim per word
  const int wpd = bs / 8;
  for (int i = threadIdx.x; i < d * wpd; i += 32 * kQaWarps) {
    const int c = i / wpd, t0 = 8 * (i % wpd);
    if (t0 + 8 <= s0 || t0 >= s1) continue;
    uint32_t w = 0, keep = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int slot = t0 + k;
      if (slot >= s0 && slot < s1) w |= (uint32_t)qa_codes[(bs + slot) * d + c] << (4 * k);
      else keep |= 0xFu << (4 * k);
    }
    uint32_t *p = reinterpret_cast<uint32_t *>(a.cache[1] + rec + q4_v_byte(t0, c, bs));
    if (keep) w |= *p & keep;
    *p = w;
  }
}

struct Q4GatherArgs {
  const uint8_t *cache[2];
  void *out[2];   // [B][n_rows][H_kv][d]
  const int32_t *block_table, *seq_lens, *start;
  int max_blocks, n_rows, H_kv, d, bs, num_blocks;
  int64_t block_stride, head_stride;   // bytes
  int32_t *status;
};

// Any head dim and block size: a thread per value.
template <typename TO>
__global__ void __launch_bounds__(256) q4_gather_kernel(const __grid_constant__ Q4GatherArgs a) {
  pdl_wait();
  pdl_trigger();
  const int i = blockIdx.x, b = blockIdx.y;
  const int L = a.seq_lens[b];
  const bool len_ok = L >= 0 && L <= a.max_blocks * a.bs;
  if (!len_ok && threadIdx.x == 0 && i == 0) atomic_or_status(a.status, SV_DEV_BAD_SEQ_LEN);
  const int64_t pos = (int64_t)a.start[b] + i;
  int phys = -1;
  if (len_ok && pos >= 0 && pos < L) {
    phys = a.block_table[(int64_t)b * a.max_blocks + pos / a.bs];
    if (phys < 0 || phys >= a.num_blocks) {
      if (threadIdx.x == 0) atomic_or_status(a.status, SV_DEV_BAD_BLOCK);
      phys = -1;
    }
  }
  const int slot = (int)(pos % a.bs);
  const int64_t row = ((int64_t)b * a.n_rows + i) * a.H_kv;
  for (int e = threadIdx.x; e < 2 * a.H_kv * a.d; e += blockDim.x) {
    const int kv = e / (a.H_kv * a.d), r = e - kv * a.H_kv * a.d;
    const int g = r / a.d, c = r - g * a.d;
    float v = 0.f;
    if (phys >= 0) {
      const uint8_t *rec = a.cache[kv] + (int64_t)phys * a.block_stride + (int64_t)g * a.head_stride;
      const int code = kv ? (rec[q4_v_byte(slot, c, a.bs)] >> (4 * (slot & 1))) & 15
                          : (rec[q4_k_byte(slot, c, a.d)] >> (4 * (c & 1))) & 15;
      const __half *pr = reinterpret_cast<const __half *>(rec + q4_code_bytes(a.d, a.bs)) + 2 * slot;
      v = fmaf((float)code, __half2float(pr[0]), __half2float(pr[1]));
    }
    TO *o = static_cast<TO *>(a.out[kv]) + (row + g) * a.d + c;
    if constexpr (sizeof(TO) == 4) *o = v;
    else *o = __float2bfloat16_rn(v);
  }
}

template <typename TIn, int NE>
sv_status launch_append_q4(const Q4AppendArgs &a, int B, cudaStream_t s) {
  const int pages = (a.n_new + a.bs - 2) / a.bs + 1;
  const bool vec = aligned(a.src[0], 8) && aligned(a.src[1], 8);
  launch_k(q4_append_kernel<TIn, NE>, dim3(pages, a.H_kv, B), dim3(32 * kQaWarps), (size_t)2 * a.bs * 32 * NE, s, 1, a,
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
  Q4GatherArgs a = {};
  const sv_status rc = q4_check("kv_block_gather_q4", k_cache, v_cache, layout, H_kv, d_head, block_size,
                                &a.block_stride, &a.head_stride);
  if (rc != SV_OK) return rc;
  if (B == 0 || n_rows == 0) return ok();
  a.cache[0] = static_cast<const uint8_t *>(k_cache); a.cache[1] = static_cast<const uint8_t *>(v_cache);
  a.out[0] = k_out; a.out[1] = v_out; a.block_table = block_table; a.seq_lens = seq_lens; a.start = start;
  a.max_blocks = max_blocks_per_seq; a.n_rows = n_rows; a.H_kv = H_kv; a.d = d_head; a.bs = block_size;
  a.num_blocks = num_blocks; a.status = dev_status;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const dim3 grid(n_rows, B);
  if (out_dtype == SV_F32) launch_k(q4_gather_kernel<float>, grid, dim3(256), 0, s, 1, a);
  else launch_k(q4_gather_kernel<__nv_bfloat16>, grid, dim3(256), 0, s, 1, a);
  return check_launch("kv_block_gather_q4 launch");
}
