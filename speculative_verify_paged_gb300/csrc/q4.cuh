// The 4-bit page record and the span of keys a windowed call reads, shared by
// the 4-bit append / read-back kernels and the attention kernels.
//
// Record of one (block, kv head) of a 4-bit pool: block_size * d / 2 bytes of
// codes, then block_size pairs (scale, minimum) of f16, one per slot. A value
// is code * scale + minimum, code in 0..15.
//   K: slot-major, d / 2 bytes a slot (byte i: head dim 2i low, 2i + 1 high).
//      With d a multiple of 128 the 16-byte chunk c of slot s is stored at
//      chunk c ^ ((s >> 1) & 3): eight threads that each read one chunk of
//      their own slot, as the attention kernel does, then touch eight
//      different 16-byte columns of shared memory.
//   V: dim-major, block_size / 2 bytes a head dim (byte i: slot 2i low,
//      2i + 1 high), so that a thread that owns a head dim reads the codes of
//      a block's keys in one piece.
#pragma once

#include "sv_common.cuh"

namespace sv {

__host__ __device__ inline int q4_code_bytes(int d, int bs) { return bs * d / 2; }
__host__ __device__ inline int q4_record_bytes(int d, int bs) { return bs * d / 2 + 4 * bs; }

// Byte of slot `slot`, head dim c (low four bits for even c) in a K record.
__host__ __device__ inline int q4_k_byte(int slot, int c, int d) {
  int chunk = c >> 5;
  if (d % 128 == 0) chunk ^= (slot >> 1) & 3;
  return slot * (d >> 1) + (chunk << 4) + ((c >> 1) & 15);
}
// Byte of slot `slot` (low four bits for even slots), head dim c in a V record.
__host__ __device__ inline int q4_v_byte(int slot, int c, int bs) { return c * (bs >> 1) + (slot >> 1); }

// The keys a call reads of a sequence of length L. Without a window that is
// every key. With one, query position p sees t <= p with t > p - window or
// t < sinks, so the blocks between the last sink block and the first block the
// oldest query's window reaches are skipped: block v of the span is block v of
// the sequence for v < nsb, else block v + skip. In these span coordinates
// (key t becomes t - 16 skip behind the gap) everything else is unchanged: the
// length is L - skip * bs, the diagonal moves with it, and key t is visible to
// the query at p iff t <= p and (t < sinks or t > p - window): a gap means that
// the sink blocks end before it, and keys of the last sink block past `sinks`
// lie before every window.
struct KeySpan {
  int L;      // length in span coordinates
  int nblk;   // blocks of the span
  int nsb;    // blocks before the gap
  int skip;   // blocks left out
};

__host__ __device__ inline KeySpan key_span(int L, int n_new, int window, int sinks, int bs) {
  KeySpan s;
  s.nblk = (L + bs - 1) / bs;
  s.nsb = 0;
  s.skip = 0;
  if (window > 0) {
    const int lo = L - n_new - window + 1;   // first key of the oldest query's window
    const int wb0 = lo > 0 ? lo / bs : 0;
    const int sb = sinks > 0 ? (int)(((int64_t)sinks + bs - 1) / bs) : 0;
    s.nsb = sb < wb0 ? sb : wb0;
    s.skip = wb0 - s.nsb;
    s.nblk -= s.skip;
  }
  s.L = L - s.skip * bs;
  return s;
}

// Most blocks a span can have (host: sizes grids and workspaces).
inline int span_blocks_max(int max_blocks, int n_new, int window, int sinks, int bs) {
  if (window <= 0) return max_blocks;
  const int64_t n = ((int64_t)sinks + bs - 1) / bs + ((int64_t)window + n_new - 2) / bs + 2;
  return (int)(n < max_blocks ? n : max_blocks);
}

// Positions and lengths are 32-bit integers and tiles run past the end: the
// entry points here take tables of less than 2^30 tokens a sequence.
inline bool capacity_ok(int max_blocks, int bs) { return (int64_t)max_blocks * bs < (1ll << 30); }

// Marks a 4-bit pool inside the library (the pools carry their own scales, so
// no entry point takes it as an element type).
constexpr sv_dtype kQ4 = static_cast<sv_dtype>(4);

// Checks the sizes, alignment and layout of 4-bit pools and gives the strides
// of their records in bytes.
sv_status q4_check(const char *what, const void *k_cache, const void *v_cache, const sv_kv_layout *layout, int H_kv,
                   int d_head, int block_size, int64_t *block_stride, int64_t *head_stride);

// spec_verify_attn_q4 on the CUDA-core kernel (attn.cu), for every shape and
// type, with all its argument checks.
sv_status attn_cuda_core_q4(const void *q, sv_dtype q_dtype, const void *k_cache, const void *v_cache,
                            const sv_kv_layout *layout, const int32_t *block_table, int max_blocks_per_seq,
                            const int32_t *seq_lens, int B, int n_new, int H_q, int H_kv, int d_head, int block_size,
                            int num_blocks, float softmax_scale, int window, int sinks, void *out, sv_dtype out_dtype,
                            void *workspace, size_t workspace_bytes, int32_t *dev_status, sv_stream_t stream);

}  // namespace sv
