// spec_rope: rotary positions of the new queries and keys of a verify round,
// and the frequencies of the usual ways to stretch a context.
//
// Pair i of the r rotated dims of a row at position p turns by p w_i, times m:
//   (a, b) -> m (a cos - b sin, b cos + a sin).
// The angle is taken in turns: w_i / (2 pi) as a 64-bit fixed-point fraction,
// times p modulo 2^64, is the fraction of a turn to 2^-33 at any 32-bit
// position, from one integer product; its upper 32 bits go to sincospif. (In
// f32 the angle of position 131071 is off by up to 2^-8 for w_0 = 1.)
#include <algorithm>
#include <cmath>
#include <cstring>

#include "sv_common.cuh"

namespace sv {
namespace {

constexpr double kTwoPi = 6.283185307179586476925286766559;

struct RopeArgs {
  const void *src[2];      // queries, keys
  void *dst[2];
  int64_t seq[4], row[4], head[4];   // strides in elements: src of queries and keys, then dst
  int H[2];
  const int32_t *positions, *seq_lens;
  int n_new, d, r, offset;
  int units, rotated;      // pieces of work of a head, the first `rotated` of them pairs
  unsigned magic;          // floor(x / units) = x magic >> 32 (0: units is 1)
  int heads;               // of a CTA
  bool copy[2];            // the dims that stay are copied
  float m;
  int32_t *status;
  unsigned long long turns[SV_ROPE_MAX_DIM / 2];
};

template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }

template <typename T, int V>
__device__ __forceinline__ void load_v(const T *p, T (&x)[V]) {
  if constexpr (V > 1) *reinterpret_cast<uint4 *>(x) = *reinterpret_cast<const uint4 *>(p);
  else x[0] = p[0];
}
template <typename T, int V>
__device__ __forceinline__ void store_v(T *p, const T (&x)[V]) {
  if constexpr (V > 1) *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(x);
  else p[0] = x[0];
}

// A CTA takes `heads` heads (queries first, then keys) of one row: the cosines
// and sines of the row once, a thread a pair, then pieces of V pairs (two
// 16-byte vectors, or two elements where something is not aligned to 16 bytes)
// and of V dims that stay.
constexpr int kRopeThreads = 256;
template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ __align__(16) float s_cos[SV_ROPE_MAX_DIM / 2], s_sin[SV_ROPE_MAX_DIM / 2];
  pdl_trigger();
  const int64_t rowi = blockIdx.x;
  const int b = (int)(rowi / a.n_new), j = (int)(rowi % a.n_new);
  int pos = 0;
  bool ok = true;
  // (positions may be what the kernel before writes; the lengths never are)
  if (!a.positions) {
    const int L = a.seq_lens[b];
    ok = L >= a.n_new;
    pos = L - a.n_new + j;
  }
  pdl_wait();
  if (a.positions) pos = a.positions[rowi];
  if (!ok) {
    if (threadIdx.x == 0 && blockIdx.y == 0) atomic_or_status(a.status, SV_DEV_BAD_SEQ_LEN);
    return;
  }
  for (int i = threadIdx.x; i < a.r / 2; i += kRopeThreads) {
    const unsigned long long turn = (unsigned long long)(long long)pos * a.turns[i];
    float s, c;
    sincospif((float)(int)(turn >> 32) * 0x1p-31f, &s, &c);
    s_cos[i] = c * a.m;
    s_sin[i] = s * a.m;
  }
  __syncthreads();
  const int h0 = blockIdx.y * a.heads, n = min(a.heads, a.H[0] + a.H[1] - h0) * a.units;
  for (int x = threadIdx.x; x < n; x += kRopeThreads) {
    const int hh = a.magic ? (int)__umulhi((unsigned)x, a.magic) : x, u = x - hh * a.units;
    int h = h0 + hh;
    const int w = h >= a.H[0] ? 1 : 0;
    if (w) h -= a.H[0];
    const T *src = static_cast<const T *>(a.src[w]) + b * a.seq[w] + j * a.row[w] + h * a.head[w];
    T *dst = static_cast<T *>(a.dst[w]) + b * a.seq[2 + w] + j * a.row[2 + w] + h * a.head[2 + w];
    alignas(16) T lo[V], hi[V];
    if (u < a.rotated) {
      const int i = u * V;   // first pair
      const int at = a.offset + (INTER ? 2 * i : i), step = INTER ? V : a.r / 2;
      load_v<T, V>(src + at, lo);
      load_v<T, V>(src + at + step, hi);
#pragma unroll
      for (int k = 0; k < V; ++k) {
        // pair k: interleaved, elements 2k and 2k + 1 of the 2 V in a row
        T &ta = !INTER ? lo[k] : 2 * k < V ? lo[2 * k] : hi[2 * k - V];
        T &tb = !INTER ? hi[k] : 2 * k + 1 < V ? lo[2 * k + 1] : hi[2 * k + 1 - V];
        const float xa = to_f32(ta), xb = to_f32(tb), c = s_cos[i + k], s = s_sin[i + k];
        ta = from_f32<T>(xa * c - xb * s);
        tb = from_f32<T>(xb * c + xa * s);
      }
      store_v<T, V>(dst + at, lo);
      store_v<T, V>(dst + at + step, hi);
    } else if (a.copy[w]) {
      int at = (u - a.rotated) * V;
      if (at >= a.offset) at += a.r;
      load_v<T, V>(src + at, lo);
      store_v<T, V>(dst + at, lo);
    }
  }
}

template <typename T>
sv_status launch_rope(RopeArgs &a, int B, bool inter, bool vec, cudaStream_t s) {
  constexpr int V = 16 / (int)sizeof(T);
  const int v = vec ? V : 1;
  a.rotated = a.r / 2 / v;
  a.units = a.rotated + (a.copy[0] || a.copy[1] ? (a.d - a.r) / v : 0);
  a.magic = a.units > 1 ? (unsigned)(0x100000000ull / (unsigned)a.units + 1) : 0;
  const int H = a.H[0] + a.H[1];
  const int64_t rows = (int64_t)B * a.n_new;
  // Many rows: a CTA takes all heads of a row (up to 2^14 pieces). Few: a piece
  // or two a thread, so that one token's heads spread over the SMs.
  int64_t per = rows >= 1024 ? (1 << 14) : 2 * kRopeThreads;
  a.heads = (int)std::max<int64_t>(1, std::min<int64_t>(H, per / a.units));
  const dim3 grid((unsigned)rows, (unsigned)((H + a.heads - 1) / a.heads));
  if (inter) {
    if (vec) launch_k(rope_kernel<T, V, true>, grid, dim3(kRopeThreads), 0, s, 1, a);
    else launch_k(rope_kernel<T, 1, true>, grid, dim3(kRopeThreads), 0, s, 1, a);
  } else {
    if (vec) launch_k(rope_kernel<T, V, false>, grid, dim3(kRopeThreads), 0, s, 1, a);
    else launch_k(rope_kernel<T, 1, false>, grid, dim3(kRopeThreads), 0, s, 1, a);
  }
  return check_launch("spec_rope launch");
}

bool rope_ok(const sv_rope *r) { return r && r->rotary_dim >= 2 && r->rotary_dim % 2 == 0 && r->rotary_dim <= SV_ROPE_MAX_DIM; }

}  // namespace
}  // namespace sv

extern "C" sv_status sv_rope_init(sv_rope *rope, int rotary_dim, double theta) {
  using namespace sv;
  if (!rope) return fail(SV_ERR_INVALID_ARG, "sv_rope_init: null pointer argument");
  if (rotary_dim < 2 || rotary_dim % 2 || rotary_dim > SV_ROPE_MAX_DIM)
    return fail(SV_ERR_INVALID_ARG, "sv_rope_init: rotary_dim must be even and in 2..%d", SV_ROPE_MAX_DIM);
  if (!(theta > 1.0) || !std::isfinite(theta)) return fail(SV_ERR_INVALID_ARG, "sv_rope_init: theta must be finite and above 1");
  memset(rope, 0, sizeof(*rope));
  rope->rotary_dim = rotary_dim;
  rope->scale = 1.f;
  for (int i = 0; i < rotary_dim / 2; ++i) rope->inv_freq[i] = std::pow(theta, -2.0 * i / rotary_dim);
  return ok();
}

extern "C" sv_status sv_rope_scale_linear(sv_rope *rope, double factor) {
  using namespace sv;
  if (!rope_ok(rope)) return fail(SV_ERR_INVALID_ARG, "sv_rope_scale_linear: not an initialised sv_rope");
  if (!(factor > 0.0) || !std::isfinite(factor)) return fail(SV_ERR_INVALID_ARG, "sv_rope_scale_linear: factor must be finite and > 0");
  for (int i = 0; i < rope->rotary_dim / 2; ++i) rope->inv_freq[i] /= factor;
  return ok();
}

extern "C" sv_status sv_rope_scale_llama3(sv_rope *rope, double factor, double low_freq_factor, double high_freq_factor,
                                          double original_length) {
  using namespace sv;
  if (!rope_ok(rope)) return fail(SV_ERR_INVALID_ARG, "sv_rope_scale_llama3: not an initialised sv_rope");
  if (!(factor > 0.0) || !std::isfinite(factor) || !(low_freq_factor > 0.0) || !(high_freq_factor > low_freq_factor) ||
      !std::isfinite(high_freq_factor) || !(original_length > 0.0) || !std::isfinite(original_length))
    return fail(SV_ERR_INVALID_ARG, "sv_rope_scale_llama3: factor > 0, 0 < low_freq_factor < high_freq_factor and original_length > 0 are needed");
  for (int i = 0; i < rope->rotary_dim / 2; ++i) {
    const double w = rope->inv_freq[i], turns = original_length * w / kTwoPi;   // over the original context
    const double keep = std::fmin(1.0, std::fmax(0.0, (turns - low_freq_factor) / (high_freq_factor - low_freq_factor)));
    rope->inv_freq[i] = w * keep + w / factor * (1.0 - keep);
  }
  return ok();
}

extern "C" sv_status sv_rope_scale_yarn(sv_rope *rope, double theta, double factor, double beta_fast, double beta_slow,
                                        double original_length, double attention_factor) {
  using namespace sv;
  if (!rope_ok(rope)) return fail(SV_ERR_INVALID_ARG, "sv_rope_scale_yarn: not an initialised sv_rope");
  if (!(theta > 1.0) || !std::isfinite(theta) || !(factor > 0.0) || !std::isfinite(factor) || !(beta_slow > 0.0) ||
      !(beta_fast >= beta_slow) || !std::isfinite(beta_fast) || !(original_length > 0.0) || !std::isfinite(original_length) ||
      !std::isfinite(attention_factor) || attention_factor < 0.0)
    return fail(SV_ERR_INVALID_ARG, "sv_rope_scale_yarn: theta > 1, factor > 0, 0 < beta_slow <= beta_fast, original_length > 0 and attention_factor >= 0 are needed");
  const int r = rope->rotary_dim;
  // the pair that makes so many turns over the original context
  auto pair_of = [&](double turns) { return r * std::log(original_length / (turns * kTwoPi)) / (2.0 * std::log(theta)); };
  const double lo = std::fmax(std::floor(pair_of(beta_fast)), 0.0);
  double hi = std::fmin(std::ceil(pair_of(beta_slow)), r - 1.0);
  if (hi == lo) hi += 0.001;
  for (int i = 0; i < r / 2; ++i) {
    const double w = rope->inv_freq[i], ramp = std::fmin(1.0, std::fmax(0.0, (i - lo) / (hi - lo)));
    rope->inv_freq[i] = w / factor * ramp + w * (1.0 - ramp);
  }
  rope->scale *= (float)(attention_factor > 0.0 ? attention_factor : factor > 1.0 ? 0.1 * std::log(factor) + 1.0 : 1.0);
  return ok();
}

extern "C" sv_status spec_rope(const void *q, void *q_out, const void *k, void *k_out, sv_dtype dtype,
                               const sv_rope_rows *q_rows, const sv_rope_rows *q_out_rows, const sv_rope_rows *k_rows,
                               const sv_rope_rows *k_out_rows, const sv_rope *rope, const int32_t *positions,
                               const int32_t *seq_lens, int B, int n_new, int H_q, int H_kv, int d, int32_t *dev_status,
                               sv_stream_t stream) {
  using namespace sv;
  if (B < 0 || n_new < 1 || H_q < 0 || H_kv < 0 || H_q + (int64_t)H_kv < 1 || d < 2)
    return fail(SV_ERR_INVALID_ARG, "spec_rope: bad sizes");
  if ((H_q && (!q || !q_out)) || (H_kv && (!k || !k_out)) || (!positions && !seq_lens))
    return fail(SV_ERR_INVALID_ARG, "spec_rope: null pointer argument");
  if (!rope_ok(rope)) return fail(SV_ERR_INVALID_ARG, "spec_rope: not an initialised sv_rope");
  if (rope->offset < 0 || (int64_t)rope->offset + rope->rotary_dim > d)
    return fail(SV_ERR_INVALID_ARG, "spec_rope: dims %d .. %lld of rows of %d", rope->offset, (long long)rope->offset + rope->rotary_dim - 1, d);
  if (!std::isfinite(rope->scale)) return fail(SV_ERR_INVALID_ARG, "spec_rope: the scale must be finite");
  if (dtype != SV_F32 && dtype != SV_BF16 && dtype != SV_F16) return fail(SV_ERR_UNSUPPORTED, "spec_rope: rows must be f32, bf16 or f16");
  if (d > 65535 || H_q + (int64_t)H_kv > 65535) return fail(SV_ERR_UNSUPPORTED, "spec_rope: d or the heads too large");
  if ((int64_t)B * n_new >= (1ll << 31)) return fail(SV_ERR_UNSUPPORTED, "spec_rope: too many rows");
  if (B == 0) return ok();
  RopeArgs a;
  memset(&a, 0, sizeof(a));
  const int es = dtype_bytes(dtype);
  a.H[0] = H_q; a.H[1] = H_kv;
  a.src[0] = q; a.src[1] = k; a.dst[0] = q_out; a.dst[1] = k_out;
  const sv_rope_rows *rows[4] = {q_rows, k_rows, q_out_rows, k_out_rows};
  const int V = 16 / es;
  const bool inter = rope->interleaved != 0;
  bool vec = rope->offset % V == 0 && d % V == 0 && (rope->rotary_dim / 2) % V == 0;
  for (int t = 0; t < 4; ++t) {
    const int H = a.H[t & 1];
    if (!H) continue;
    if (rows[t] && (rows[t]->head_stride < 0 || rows[t]->row_stride < 0 || rows[t]->seq_stride < 0))
      return fail(SV_ERR_INVALID_ARG, "spec_rope: negative strides");
    a.head[t] = rows[t] ? rows[t]->head_stride : d;
    a.row[t] = rows[t] ? rows[t]->row_stride : (int64_t)H * d;
    a.seq[t] = rows[t] ? rows[t]->seq_stride : (int64_t)n_new * H * d;
    // rows that are written must not overlap
    if (t >= 2 && ((H > 1 && a.head[t] < d) || (n_new > 1 && a.row[t] < d) || (B > 1 && a.seq[t] < d)))
      return fail(SV_ERR_INVALID_ARG, "spec_rope: output strides smaller than d");
    vec = vec && a.head[t] % V == 0 && a.row[t] % V == 0 && a.seq[t] % V == 0 && aligned(t < 2 ? a.src[t] : a.dst[t - 2], 16);
  }
  for (int w = 0; w < 2; ++w) {
    const bool same = a.src[w] == a.dst[w];
    if (a.H[w] && same && (a.head[w] != a.head[2 + w] || a.row[w] != a.row[2 + w] || a.seq[w] != a.seq[2 + w]))
      return fail(SV_ERR_INVALID_ARG, "spec_rope: rows rotated in place need the same strides on both sides");
    a.copy[w] = a.H[w] && !same;
  }
  a.positions = positions; a.seq_lens = seq_lens; a.n_new = n_new;
  a.d = d; a.r = rope->rotary_dim; a.offset = rope->offset; a.m = rope->scale; a.status = dev_status;
  for (int i = 0; i < a.r / 2; ++i) {
    double f = rope->inv_freq[i] / kTwoPi;   // turns a position
    if (!std::isfinite(f)) return fail(SV_ERR_INVALID_ARG, "spec_rope: inv_freq[%d] is not finite", i);
    f = (f - std::floor(f)) * 0x1p64;
    a.turns[i] = f < 0x1p64 ? (unsigned long long)f : 0;
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == SV_F32) return launch_rope<float>(a, B, inter, vec, s);
  if (dtype == SV_BF16) return launch_rope<__nv_bfloat16>(a, B, inter, vec, s);
  return launch_rope<__half>(a, B, inter, vec, s);
}
