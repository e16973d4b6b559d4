// spec_verify_attn_q8: paged GQA verify attention over an 8-bit block-scaled
// cache (page layout: q8.cuh).
#include <algorithm>

#include "q8.cuh"

using namespace sv;

extern "C" size_t spec_verify_attn_q8_workspace_size(int B, int n_new, int H_q, int H_kv, int d_head,
                                                     int max_blocks_per_seq, int block_size, int window, int sinks) {
  return spec_verify_attn_window_workspace_size(B, n_new, H_q, H_kv, d_head, max_blocks_per_seq, block_size, window,
                                                sinks);
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
  return attn_cuda_core_q8(q, q_dtype, k_cache, v_cache, layout, block_table, max_blocks_per_seq, seq_lens, B, n_new,
                           H_q, H_kv, d_head, block_size, num_blocks, softmax_scale, window, sinks, out, out_dtype,
                           workspace, workspace_bytes, dev_status, stream);
}
