// The 8-bit page, shared by the append / read-back kernels and the attention
// kernels.
//
// Page of one block of an 8-bit pool: H_kv * block_size * d e4m3 codes
// ([H_kv][block_size][d], as in the pools of whole elements), then H_kv f32
// scales, padded to a multiple of 128 bytes, so that the codes of every block
// start on a cache line. A value is code * scale.
// The append writes scales that are powers of two: e4m3 keeps its four
// significant bits whatever the scale, so nothing is lost against a scale of
// amax / 448, and codes whose block's scale grows later are moved exactly, but
// for those that become subnormal.
#pragma once

#include "q4.cuh"

namespace sv {

constexpr int kQ8MaxExp = 32;                // scales lie in 2^-32 .. 2^32
constexpr float kQ8MinScale = 0x1p-32f, kQ8MaxScale = 0x1p32f;

__host__ __device__ inline int64_t q8_scale_offset(int H_kv, int d, int bs) { return (int64_t)H_kv * bs * d; }
__host__ __device__ inline int64_t q8_page_bytes(int H_kv, int d, int bs) {
  return (q8_scale_offset(H_kv, d, bs) + 4 * (int64_t)H_kv + 127) / 128 * 128;
}

// A scale as every reader takes it (a page that was never written holds zeros;
// fmaxf drops a NaN).
__device__ __forceinline__ float q8_scale(float s) { return fminf(fmaxf(s, kQ8MinScale), kQ8MaxScale); }

// Marks an 8-bit block-scaled pool inside the library.
constexpr sv_dtype kQ8 = static_cast<sv_dtype>(5);

// Checks the sizes, alignment and layout of 8-bit pools and gives the stride
// of their pages in bytes.
sv_status q8_check(const char *what, const void *k_cache, const void *v_cache, const sv_kv_layout *layout, int H_kv,
                   int d_head, int block_size, int64_t *block_stride);

// Whether the CUDA-core kernel (attn.cu) takes R query rows a kv head.
bool attn_cuda_core_fits(int64_t R, int d_head);

// spec_verify_attn_q8 on the CUDA-core kernel, for every shape and type, with
// all its argument checks.
sv_status attn_cuda_core_q8(const void *q, sv_dtype q_dtype, const void *k_cache, const void *v_cache,
                            const sv_kv_layout *layout, const int32_t *block_table, int max_blocks_per_seq,
                            const int32_t *seq_lens, int B, int n_new, int H_q, int H_kv, int d_head, int block_size,
                            int num_blocks, float softmax_scale, int window, int sinks, void *out, sv_dtype out_dtype,
                            void *workspace, size_t workspace_bytes, int32_t *dev_status, sv_stream_t stream);

}  // namespace sv
