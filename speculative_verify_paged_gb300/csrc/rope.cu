// spec_rope: rotary positions of the new queries and keys of a verify round,
// and the frequencies of the usual ways to stretch a context.
//
// Pair i of the r rotated dims of a row at position p turns by p w_i, times m:
//   (a, b) -> m (a cos - b sin, b cos + a sin).
// The angle is taken in turns: w_i / (2 pi) as a 64-bit fixed-point fraction,
// times p modulo 2^64, is the fraction of a turn to 2^-33 at any 32-bit
// position, from one integer product; its upper 32 bits, as half turns in f32
// (rounded to 2^-26 turns), go to sincospif. The fraction needs more than a
// double holds (2^-56 of a turn a position would be 2^-25 at position 2^31): it
// is made from w_i / (2 pi) in two doubles. (In f32 the angle of position 131071
// is off by up to 2^-8 for w_0 = 1.)
#include <algorithm>
#include <cmath>
#include <cstring>
#include <utility>

#include "sv_common.cuh"

namespace sv {
namespace {

constexpr double kTwoPi = 6.283185307179586476925286766559;
constexpr double kTurn = 0.15915494309189535, kTurnLow = -9.839338337591243e-18;   // 1 / (2 pi) to 2^-110

struct RopeArgs {
  const void *src[2];      // queries, keys
  void *dst[2];
  int64_t seq[4], row[4], head[4];   // strides in elements: src of queries and keys, then dst
  int H[2];
  const int32_t *positions, *seq_lens;
  int n_new, d, r, offset;
  int units, rotated;      // pieces of work of a head, the first `rotated` of them pairs
  int lanes, side;         // threads of a head, heads side by side
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

// A CTA takes `heads` heads (queries first, then keys) of one row, in pieces: V
// pairs, or two vectors of V dims that stay (V: a 16-byte vector, or one element
// where something is not aligned to 16 bytes). A thread takes the same piece of
// every side-th head, kRopeBatch heads at a time: what a piece needs besides its
// data is worked out once (with places worked out per piece the kernel was short of
// instructions, not of bandwidth). The first batch is read before the row's cosines
// and sines are made, a thread a pair.
// Bound by memory: 32752 rows of 72 heads of 128 bf16, 64 dims rotated, 1.21 GB
// read and written, take 171 us (282 with places per piece; batches of 2 heads 188,
// of 4 181); 160 rows of 129 heads of 576, 48 MB, 13.4 us with the launch (23.7).
// By elements it is bound by their number: 36 of 128 dims of the same rows 441 us.
constexpr int kRopeThreads = 256, kRopeBatch = 3;
template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ __align__(16) float s_cos[SV_ROPE_MAX_DIM / 2], s_sin[SV_ROPE_MAX_DIM / 2];
  pdl_trigger();
  const unsigned rowi = blockIdx.x;
  const int b = (int)(rowi / (unsigned)a.n_new), j = (int)(rowi % (unsigned)a.n_new);
  const int hh = (int)(threadIdx.x / (unsigned)a.lanes);
  int u = (int)threadIdx.x - hh * a.lanes;
  const int H_q = a.H[0], h0 = blockIdx.y * a.heads + hh, h1 = min((blockIdx.y + 1) * a.heads, H_q + a.H[1]);
  const T *src[2];
  T *dst[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {   // (of head 0, counted over both)
    src[w] = static_cast<const T *>(a.src[w]) + b * a.seq[w] + j * a.row[w] - (w ? H_q * a.head[1] : 0);
    dst[w] = static_cast<T *>(a.dst[w]) + b * a.seq[2 + w] + j * a.row[2 + w] - (w ? H_q * a.head[3] : 0);
  }
  // (positions may be what the kernel before writes; the lengths never are)
  int pos = 0;
  bool ok = true;
  if (!a.positions) {
    const int L = a.seq_lens[b];
    ok = L >= a.n_new;
    pos = L - a.n_new + j;
  }
  pdl_wait();
  if (!ok) {
    if (threadIdx.x == 0 && blockIdx.y == 0) atomic_or_status(a.status, SV_DEV_BAD_SEQ_LEN);
    return;
  }
  if (a.positions) pos = a.positions[rowi];
  const int stay = a.d - a.r;
  auto dim = [&](int k) { return k < a.offset ? k : k + a.r; };   // of the k-th that stays
  alignas(16) T lo[kRopeBatch][V], hi[kRopeBatch][V];
  int at0 = 0, at1 = 0, h = h0;
  bool two = true;
  auto place = [&] {   // where a piece's two vectors are in its head
    if (u < a.rotated) {
      at0 = a.offset + u * (INTER ? 2 * V : V);
      at1 = at0 + (INTER ? V : a.r / 2);
    } else {
      const int c = (u - a.rotated) * V, c1 = c + (a.units - a.rotated) * V;
      at0 = dim(c);
      at1 = dim(c1);
      two = c1 < stay;
    }
  };
  auto fetch = [&] {
#pragma unroll
    for (int k = 0; k < kRopeBatch; ++k) {
      const int head = h + k * a.side;
      if (head >= h1) break;
      const bool key = head >= H_q;
      if (u >= a.rotated && !a.copy[key]) continue;
      const T *p = (key ? src[1] : src[0]) + head * (key ? a.head[1] : a.head[0]);
      load_v<T, V>(p + at0, lo[k]);
      if (two) load_v<T, V>(p + at1, hi[k]);
    }
  };
  bool live = hh < a.side && u < a.units && h < h1;
  if (live) {
    place();
    fetch();
  }
  for (int i = threadIdx.x; i < a.r / 2; i += blockDim.x) {
    const unsigned long long turn = (unsigned long long)(long long)pos * a.turns[i];
    float s, c;
    sincospif((float)(int)(turn >> 32) * 0x1p-31f, &s, &c);
    s_cos[i] = c * a.m;
    s_sin[i] = s * a.m;
  }
  __syncthreads();
  while (live) {
    float c[V], s[V];
    if (u < a.rotated) {
      if constexpr (V > 1) {
#pragma unroll
        for (int e = 0; e < V; e += 4) {
          *reinterpret_cast<float4 *>(c + e) = *reinterpret_cast<const float4 *>(&s_cos[u * V + e]);
          *reinterpret_cast<float4 *>(s + e) = *reinterpret_cast<const float4 *>(&s_sin[u * V + e]);
        }
      } else {
        c[0] = s_cos[u];
        s[0] = s_sin[u];
      }
    }
#pragma unroll
    for (int k = 0; k < kRopeBatch; ++k) {
      const int head = h + k * a.side;
      if (head >= h1) break;
      const bool key = head >= H_q;
      if (u < a.rotated) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          // pair e: interleaved, elements 2e and 2e + 1 of the 2 V in a row
          T &ta = !INTER ? lo[k][e] : 2 * e < V ? lo[k][2 * e] : hi[k][2 * e - V];
          T &tb = !INTER ? hi[k][e] : 2 * e + 1 < V ? lo[k][2 * e + 1] : hi[k][2 * e + 1 - V];
          const float xa = to_f32(ta), xb = to_f32(tb);
          ta = from_f32<T>(xa * c[e] - xb * s[e]);
          tb = from_f32<T>(xb * c[e] + xa * s[e]);
        }
      } else if (!a.copy[key]) {
        continue;
      }
      T *p = (key ? dst[1] : dst[0]) + head * (key ? a.head[3] : a.head[2]);
      store_v<T, V>(p + at0, lo[k]);
      if (two) store_v<T, V>(p + at1, hi[k]);
    }
    h += kRopeBatch * a.side;
    if (h >= h1) {
      h = h0;
      u += a.lanes;
      live = u < a.units;
      if (live) place();
    }
    if (live) fetch();
  }
}

template <typename T>
sv_status launch_rope(RopeArgs &a, int B, bool inter, bool vec, cudaStream_t s) {
  constexpr int V = 16 / (int)sizeof(T);
  const int v = vec ? V : 1;
  a.rotated = a.r / 2 / v;
  a.units = a.rotated + (a.copy[0] || a.copy[1] ? ((a.d - a.r) / v + 1) / 2 : 0);
  const int H = a.H[0] + a.H[1];
  const int64_t rows = (int64_t)B * a.n_new;
  a.lanes = std::min(a.units, kRopeThreads);
  // Heads side by side as threads go, and batches in turn: all of a row's, if
  // that leaves four CTAs an SM; else as many as leave that, and a batch at most.
  const int side = kRopeThreads / a.lanes;
  const int64_t want = (rows * H + 607) / 608;   // heads of a CTA when there are four an SM
  a.heads = rows >= 608 ? H : (int)std::min<int64_t>(std::min<int64_t>(H, want), (int64_t)side * kRopeBatch);
  const int turns = (a.heads + side - 1) / side;
  a.side = (a.heads + turns - 1) / turns;
  const int threads = (a.side * a.lanes + 31) / 32 * 32;
  const dim3 grid((unsigned)rows, (unsigned)((H + a.heads - 1) / a.heads));
  if (inter) {
    if (vec) launch_k(rope_kernel<T, V, true>, grid, dim3(threads), 0, s, 1, a);
    else launch_k(rope_kernel<T, 1, true>, grid, dim3(threads), 0, s, 1, a);
  } else {
    if (vec) launch_k(rope_kernel<T, V, false>, grid, dim3(threads), 0, s, 1, a);
    else launch_k(rope_kernel<T, 1, false>, grid, dim3(threads), 0, s, 1, a);
  }
  return check_launch("spec_rope launch");
}

// The fraction of w / (2 pi) as a 64-bit one, to half a step of it for |w| up to 2^40.
unsigned long long turns_of(double w) {
  const double x = std::fabs(w), hi = x * kTurn;
  double low = std::fma(x, kTurn, -hi) + x * kTurnLow;   // hi + low = |w| / (2 pi)
  low -= std::rint(low);
  double whole;
  const double f = std::modf(hi, &whole) * 0x1p64;   // (modf: a difference with the product could be contracted)
  const unsigned long long steps = (unsigned long long)f;
  low = low * 0x1p64 + (f - (double)steps);
  const unsigned long long more = (unsigned long long)std::rint(std::fabs(low));   // at most 2^63
  const unsigned long long t = low < 0 ? steps - more : steps + more;
  return w < 0 ? 0 - t : t;
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
    // rows that are written must not overlap: by ascending stride, each beyond what those before it span
    if (t >= 2) {
      std::pair<int64_t, int64_t> by[3] = {{a.head[t], H}, {a.row[t], n_new}, {a.seq[t], B}};   // stride, count
      std::sort(by, by + 3);
      int64_t span = d;
      for (const auto &[stride, count] : by) {
        if (count < 2) continue;
        if (stride < span) return fail(SV_ERR_INVALID_ARG, "spec_rope: output rows overlap (strides %lld, %lld, %lld)",
                                       (long long)a.seq[t], (long long)a.row[t], (long long)a.head[t]);
        if (stride > (INT64_MAX - span) / (count - 1)) return fail(SV_ERR_INVALID_ARG, "spec_rope: output strides too large");
        span += (count - 1) * stride;
      }
    }
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
    if (!std::isfinite(rope->inv_freq[i])) return fail(SV_ERR_INVALID_ARG, "spec_rope: inv_freq[%d] is not finite", i);
    a.turns[i] = turns_of(rope->inv_freq[i]);
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == SV_F32) return launch_rope<float>(a, B, inter, vec, s);
  if (dtype == SV_BF16) return launch_rope<__nv_bfloat16>(a, B, inter, vec, s);
  return launch_rope<__half>(a, B, inter, vec, s);
}
