// Losses on a language model's logits, with their gradients: token
// log-probabilities, the clipped policy loss with a KL term, and the
// preference loss over paired log ratios.
//
// For row t with logits x, temperature tau and label y:
//   lp = x_y / tau - log sum_j exp(x_j / tau)
// and a loss that depends on the logits through lp alone has
//   dL/dx_j = (dL/dlp) * ([j = y] - p_j) / tau,   p_j = exp(x_j / tau) / sum.
//
// All of it is kept in base 2: with k = log2(e) / tau and any shift c,
// e_j = 2^(x_j k - c) is one FMA and one exponential, and two partial sums
// with shifts c1, c2 combine exactly by 2^(c1 - c2). Sums and shifts are fp32;
// the few operations a row does once (lp itself) are in fp64, so that lp
// carries no rounding of the shift or of the logarithm's integer part.
// Shifts are integers.
// Gradients are rounded once, into the logits' type.
//
// A row whose label is negative is not read: its log-probability is 0 and its
// gradient row is zeros, whatever the logits there hold. A label >= vocab
// makes its row NaN. A row of -inf alone has no distribution: NaN. A row of the
// type's lowest value alone is uniform.
#include "loss.h"

#include "common.cuh"

namespace ar {
namespace {

constexpr int kRowThreads = 512;
constexpr double kExpLow = 4.9e-8;

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A shift of -inf (a part of the row that is all -inf) is replaced by 0:
// its terms are then 2^-inf = 0 rather than 2^(-inf + inf).
__device__ __forceinline__ float finite_shift(float c) { return c == -INFINITY ? 0.0f : c; }

// 2^d for an integer d <= 0, exactly (0 below the normal numbers).
__device__ __forceinline__ float pow2(float d) {
  const int e = int(fmaxf(d, -127.0f)) + 127;
  return e > 0 ? __int_as_float(e << 23) : 0.0f;
}

// A running (shift, sum) pair in base 2: the value is s * 2^c. Shifts are
// integers, so that joining two pairs rounds only their sum; with shifts of any
// value every level of the joins would bring in the exponential's error, whose
// mean is not zero, and log-probabilities summed over a sequence would drift.
struct Lse {
  float c, s;
};
__device__ __forceinline__ Lse lse_join(Lse a, Lse b) {
  const float c = fmaxf(a.c, b.c), z = finite_shift(c);
  return {c, a.s * pow2(a.c - z) + b.s * pow2(b.c - z)};
}

// Sum of one row over the CTA; every thread gets the result. `part` holds one
// entry per warp.
template <int THREADS>
__device__ __forceinline__ Lse lse_block(Lse v, Lse* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    v = lse_join(v, {__shfl_xor_sync(~0u, v.c, o), __shfl_xor_sync(~0u, v.s, o)});
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
  __syncthreads();
  constexpr int W = THREADS / 32;
  v = part[threadIdx.x % W];
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1)
    v = lse_join(v, {__shfl_xor_sync(~0u, v.c, o), __shfl_xor_sync(~0u, v.s, o)});
  return v;
}

__device__ __forceinline__ double log_prob(const LossParams& p, float x_label, float k, Lse z) {
  // z.s = f * 2^e with f in [1/2, 1): the integer part of its logarithm is exact
  int e = 0;
  const float f = frexpf(z.s, &e);
  // The hardware's exponential is low by kExpLow of its value in the mean over
  // its fraction (measured over [-20, 0]), hence the sum too, but for the
  // label's own term where that dominates.
  const float own = exp2_approx(fmaf(x_label, k, -finite_shift(z.c))) / z.s;
  const double low = kExpLow * double(1.0f - own);
  const double above = double(x_label) * double(k) - double(finite_shift(z.c));  // first: both may be huge
  return (above - (double(e) + double(log2f(f)))) * p.to_ln - low;
}

// The range of a row of `n` elements starting at `base`: `head` elements up to
// the first 16-byte boundary, `vecs` whole 16-byte vectors, the rest.
template <int W, int ES>
struct RowSpan {
  int head;
  int64_t vecs;
  int tail;
  __device__ __forceinline__ RowSpan(const char* base, int64_t n) {
    const int off = int(reinterpret_cast<uintptr_t>(base) % 16) / ES;
    head = off ? W - off : 0;
    if (head > n) head = int(n);
    vecs = (n - head) / W;
    tail = int(n - head - vecs * W);
  }
  // The element outside the vectors that thread `i` takes (-1: none).
  __device__ __forceinline__ int64_t edge(int i) const {
    if (i < head) return i;
    return i - head < tail ? head + vecs * W + (i - head) : -1;
  }
};

template <bool BF16>
__device__ __forceinline__ float load_one(const char* base, int64_t e) {
  using L = Lane<BF16, false>;
  float f[1];
  L::widen(L::load(base, e), f);
  return f[0];
}
template <bool BF16>
__device__ __forceinline__ void store_one(char* base, int64_t e, float v) {
  using L = Lane<BF16, false>;
  const float f[1] = {v};
  L::store(base, e, L::narrow(f));
}
template <bool BF16>
__device__ __forceinline__ void load_vec(const char* base, int64_t e, float (&f)[Lane<BF16, true>::W]) {
  using L = Lane<BF16, true>;
  L::widen(L::load(base, e), f);
}
template <bool BF16>
__device__ __forceinline__ void store_vec(char* base, int64_t e, const float (&f)[Lane<BF16, true>::W], bool aligned) {
  using L = Lane<BF16, true>;
  if (aligned) {
    L::store(base, e, L::narrow(f));
  } else {
#pragma unroll
    for (int i = 0; i < L::W; ++i) store_one<BF16>(base, e + i, f[i]);
  }
}

// One row's gradient: d_j = up * [j = y] - up * p_j, p_j = 2^(x_j k - shift) * inv_sum.
template <bool BF16, int THREADS>
__device__ __forceinline__ void write_gradient(const LossParams& p, int64_t t, const char* x, int64_t label, float up,
                                               float k, float shift, float inv_sum) {
  constexpr int W = Lane<BF16, true>::W, ES = BF16 ? 2 : 4;
  char* d = static_cast<char*>(p.d) + t * p.dld * ES;
  const RowSpan<W, ES> span(x, p.vocab);
  const bool aligned = (reinterpret_cast<uintptr_t>(d) - reinterpret_cast<uintptr_t>(x)) % 16 == 0;
  const float g = -up * inv_sum;
  for (int64_t i = threadIdx.x; i < span.vecs; i += THREADS) {
    const int64_t e = span.head + i * W;
    float f[W];
    load_vec<BF16>(x, e, f);
#pragma unroll
    for (int w = 0; w < W; ++w) f[w] = exp2_approx(fmaf(f[w], k, -shift)) * g;
    if (label >= e && label < e + W) {
#pragma unroll
      for (int w = 0; w < W; ++w)
        if (label == e + w) f[w] += up;
    }
    store_vec<BF16>(d, e, f, aligned);
  }
  const int64_t e = span.edge(threadIdx.x);
  if (e >= 0) {
    const float v = exp2_approx(fmaf(load_one<BF16>(x, e), k, -shift)) * g;
    store_one<BF16>(d, e, label == e ? v + up : v);
  }
}

template <bool BF16, int THREADS>
__device__ __forceinline__ void write_zeros(const LossParams& p, int64_t t) {
  constexpr int W = Lane<BF16, true>::W, ES = BF16 ? 2 : 4;
  char* d = static_cast<char*>(p.d) + t * p.dld * ES;
  const RowSpan<W, ES> span(d, p.vocab);
  const float zero[W] = {};
  for (int64_t i = threadIdx.x; i < span.vecs; i += THREADS) store_vec<BF16>(d, span.head + i * W, zero, true);
  const int64_t e = span.edge(threadIdx.x);
  if (e >= 0) store_one<BF16>(d, e, 0.0f);
}

// The sum of one row.
template <bool BF16, int THREADS>
__device__ __forceinline__ Lse row_lse(const LossParams& p, const char* x, float k, Lse* part) {
  constexpr int W = Lane<BF16, true>::W, ES = BF16 ? 2 : 4;
  const RowSpan<W, ES> span(x, p.vocab);
  Lse z = {-INFINITY, 0.0f};
  for (int64_t i = threadIdx.x; i < span.vecs; i += THREADS) {
    float f[W];
    load_vec<BF16>(x, span.head + i * W, f);
    float top = f[0];
#pragma unroll
    for (int w = 1; w < W; ++w) top = fmaxf(top, f[w]);
    const float c = fmaxf(z.c, ceilf(top * k)), shift = finite_shift(c);
    float s = z.s * pow2(z.c - shift);
#pragma unroll
    for (int w = 0; w < W; ++w) s += exp2_approx(fmaf(f[w], k, -shift));
    z = {c, s};
  }
  const int64_t e = span.edge(threadIdx.x);
  if (e >= 0) {
    const float f = load_one<BF16>(x, e), c = ceilf(f * k);
    z = lse_join(z, {c, exp2_approx(fmaf(f, k, -finite_shift(c)))});
  }
  return lse_block<THREADS>(z, part);
}

// The same with the row's scale. Where x k itself is not finite (a row whose
// largest logit is near the type's lowest or highest value), two logits differ
// by 0 or by more than any exponent holds, at any scale: k = 1 serves.
template <bool BF16, int THREADS>
__device__ __forceinline__ Lse row_lse_scaled(const LossParams& p, const char* x, float& k, Lse* part) {
  k = p.k;
  Lse z = row_lse<BF16, THREADS>(p, x, k, part);
  if (isinf(z.c)) {
    k = 1.0f;
    __syncthreads();
    z = row_lse<BF16, THREADS>(p, x, k, part);
  }
  return z;
}

// ---------------------------------------------------------------- sequences

// Labelled tokens of each sequence (one CTA a sequence), the rows' weights,
// and, by the CTA that finishes last, 1 / (the loss's denominator).
__global__ void __launch_bounds__(256) count_kernel(LossParams p) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t s = blockIdx.x;
  auto bound = [&](int64_t i) {
    const int64_t v = p.seq_start == nullptr ? (i == 0 ? 0 : p.rows) : p.seq_start[i];
    return v < 0 ? int64_t(0) : v > p.rows ? p.rows : v;
  };
  const int64_t lo = bound(s), hi = bound(s + 1);
  __shared__ int warp_sum[8];
  __shared__ bool last;
  int n = 0;
  for (int64_t t = lo + threadIdx.x; t < hi; t += 256) n += p.labels[t] >= 0;
  n = __reduce_add_sync(~0u, n);
  if (threadIdx.x % 32 == 0) warp_sum[threadIdx.x / 32] = n;
  __syncthreads();
  n = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) n += warp_sum[w];
  const float weight = p.by_sequence ? 1.0f / float(max(n, 1)) : 1.0f;
  for (int64_t t = lo + threadIdx.x; t < hi; t += 256) p.row_a[t] = weight;
  if (s == 0)
    for (int64_t t = threadIdx.x; t < lo; t += 256) p.row_a[t] = 0.0f;
  if (s == p.n_seq - 1)
    for (int64_t t = hi + threadIdx.x; t < p.rows; t += 256) p.row_a[t] = 0.0f;
  if (threadIdx.x == 0) {
    p.seq_count[s] = n;
    __threadfence();
    last = atomicAdd(&p.tickets[0], 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  long long sum = 0;  // labelled tokens, or sequences that have any
  for (int64_t i = threadIdx.x; i < p.n_seq; i += 256) {
    const int c = __ldcg(&p.seq_count[i]);
    sum += p.by_sequence ? (c > 0) : c;
  }
  __shared__ long long parts[256];
  parts[threadIdx.x] = sum;
  __syncthreads();
  for (int o = 128; o > 0; o >>= 1) {
    if (threadIdx.x < o) parts[threadIdx.x] += parts[threadIdx.x + o];
    __syncthreads();
  }
  if (threadIdx.x == 0)
    p.total[0] = p.denominator > 0.0f ? 1.0f / p.denominator : 1.0f / float(parts[0] > 0 ? parts[0] : 1);
}

// Sums `n` entries of four columns (stride `pitch` between columns) in a fixed
// order, in fp64. Result in thread 0.
template <int THREADS>
__device__ void sum_columns(const float* col, int64_t pitch, int64_t n, int columns, double* shared, double (&out)[4]) {
  for (int c = 0; c < columns; ++c) {
    double a = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += THREADS) a += double(__ldcg(col + c * pitch + i));
    __syncthreads();
    shared[threadIdx.x] = a;
    __syncthreads();
    for (int o = THREADS / 2; o > 0; o >>= 1) {
      if (threadIdx.x < o) shared[threadIdx.x] += shared[threadIdx.x + o];
      __syncthreads();
    }
    out[c] = shared[0];
  }
}

// ---------------------------------------------------------------- rows

template <bool BF16, int MODE>
__global__ void __launch_bounds__(kRowThreads) rows_kernel(LossParams p) {
  constexpr int ES = BF16 ? 2 : 4;
  __shared__ Lse part[kRowThreads / 32];
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t t = blockIdx.x;
  const char* x = static_cast<const char*>(p.x) + t * p.ld * ES;
  const int64_t label = p.labels[t];
  const bool active = label >= 0;
  if (MODE == kPrefBackward) {
    if (!active) {
      write_zeros<BF16, kRowThreads>(p, t);
      return;
    }
    const float2 z = p.row_lse[t];  // the sign of 1 / sum tells the scale
    write_gradient<BF16, kRowThreads>(p, t, x, label, p.row_a[t] * p.inv_temp, z.y < 0.0f ? 1.0f : p.k, z.x,
                                      fabsf(z.y));
    return;
  }
  float terms[3] = {0.0f, 0.0f, 0.0f};
  float lp = 0.0f;
  if (!active) {
    if (MODE == kPolicy && p.d != nullptr) write_zeros<BF16, kRowThreads>(p, t);
  } else {
    const float x_label = label < p.vocab ? load_one<BF16>(x, label) : __int_as_float(0x7fffffff);
    float k;
    // (barriers inside: x_label is read before any gradient is written)
    const Lse z = row_lse_scaled<BF16, kRowThreads>(p, x, k, part);
    const double exact_lp = log_prob(p, x_label, k, z);
    lp = float(exact_lp);
    const float shift = finite_shift(z.c);
    if (MODE == kPrefForward && threadIdx.x == 0) {
      // the log ratio before lp is rounded: sequences sum hundreds of them
      p.row_terms[t] = float(exact_lp - double(p.ref_logp[t]));
      p.row_lse[t] = make_float2(shift, copysignf(1.0f / z.s, k == p.k ? 1.0f : -1.0f));
    }
    const float weight = MODE == kPolicy ? p.row_a[t] : 0.0f;
    if (MODE == kPolicy && weight == 0.0f) {  // outside every sequence
      if (p.d != nullptr) write_zeros<BF16, kRowThreads>(p, t);
    } else if (MODE == kPolicy) {
      const float adv = p.adv[t];
      const float ratio = expf(lp - p.old_logp[t]);
      const float free = ratio * adv;
      const float held = (ratio < p.lo ? p.lo : ratio > p.hi ? p.hi : ratio) * adv;  // NaN stays NaN
      const float w = weight * p.total[0];
      float slope = free <= held ? -free : free > held ? 0.0f : free;
      terms[0] = -w * (free < held || free != free ? free : held);
      terms[2] = held < free ? w : 0.0f;
      if (p.ref_logp != nullptr) {
        const float back = p.ref_logp[t] - lp;
        const float grow = expm1f(back);
        terms[1] = w * (grow - back);
        slope -= p.kl * grow;
      }
      if (p.d != nullptr) {
        const float up = w * slope * p.grad_scale * p.inv_temp;
        write_gradient<BF16, kRowThreads>(p, t, x, label, label < p.vocab ? up : __int_as_float(0x7fffffff), k, shift,
                                          1.0f / z.s);
      }
    }
  }
  if (threadIdx.x == 0) p.logp[t] = lp;
  if (MODE != kPolicy) return;
  __shared__ bool last;
  __shared__ double sums[kRowThreads];
  if (threadIdx.x == 0) {
    for (int c = 0; c < 3; ++c) p.row_terms[c * p.rows + t] = terms[c];
    __threadfence();
    last = atomicAdd(&p.tickets[1], 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  double out[4];
  sum_columns<kRowThreads>(p.row_terms, p.rows, p.rows, 3, sums, out);
  if (threadIdx.x == 0) {
    p.stats[0] = float(out[0] + double(p.kl) * out[1]);
    p.stats[1] = float(out[0]);
    p.stats[2] = float(out[1]);
    p.stats[3] = float(out[2]);
  }
}

// ---------------------------------------------------------------- pairs

// One CTA a pair: the log ratios of its two sequences, the loss of the pair
// and the coefficient of each of its rows.
__global__ void __launch_bounds__(256) pair_kernel(LossParams p) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t pairs = p.n_seq / 2, i = blockIdx.x;
  __shared__ double sums[256];
  __shared__ int counts[8];
  __shared__ bool last;
  auto bound = [&](int64_t s) {
    const int64_t v = p.seq_start[s];
    return v < 0 ? int64_t(0) : v > p.rows ? p.rows : v;
  };
  double ratio[2];
  float over[2];
  for (int h = 0; h < 2; ++h) {
    const int64_t lo = bound(2 * i + h), hi = bound(2 * i + h + 1);
    double a = 0.0;
    int n = 0;
    for (int64_t t = lo + threadIdx.x; t < hi; t += 256)
      if (p.labels[t] >= 0) {
        a += double(p.row_terms[t]);
        ++n;
      }
    __syncthreads();
    sums[threadIdx.x] = a;
    n = __reduce_add_sync(~0u, n);
    if (threadIdx.x % 32 == 0) counts[threadIdx.x / 32] = n;
    __syncthreads();
    for (int o = 128; o > 0; o >>= 1) {
      if (threadIdx.x < o) sums[threadIdx.x] += sums[threadIdx.x + o];
      __syncthreads();
    }
    n = 0;
    for (int w = 0; w < 8; ++w) n += counts[w];
    over[h] = p.normalize ? float(max(n, 1)) : 1.0f;
    ratio[h] = sums[0] / double(over[h]);
  }
  const double z = double(p.beta) * (ratio[0] - ratio[1]);
  double loss, slope;
  if (p.square) {
    const double off = z - double(p.target);
    loss = off * off;
    slope = 2.0 * off;
  } else {
    // log1p(e^-|z|) serves both signs of z
    const double tail = log1p(exp(-fabs(z))), up = z > 0.0 ? z : 0.0, down = z < 0.0 ? -z : 0.0;
    const double eps = double(p.smooth);
    loss = (1.0 - eps) * (tail + down) + eps * (tail + up);
    slope = -(1.0 - eps) / (1.0 + exp(z)) + eps / (1.0 + exp(-z));
    if (z != z) loss = slope = z;
  }
  const double count = p.denominator > 0.0f ? double(p.denominator) : double(pairs);
  for (int h = 0; h < 2; ++h) {
    const int64_t lo = bound(2 * i + h), hi = bound(2 * i + h + 1);
    const float c = float((h ? -1.0 : 1.0) * slope * double(p.beta) / count / double(over[h]) * double(p.grad_scale));
    for (int64_t t = lo + threadIdx.x; t < hi; t += 256) p.row_a[t] = c;
    if (h == 0 && i == 0)
      for (int64_t t = threadIdx.x; t < lo; t += 256) p.row_a[t] = 0.0f;
    if (h == 1 && i == pairs - 1)
      for (int64_t t = hi + threadIdx.x; t < p.rows; t += 256) p.row_a[t] = 0.0f;
  }
  if (threadIdx.x == 0) {
    p.ratios[2 * i] = float(ratio[0]);
    p.ratios[2 * i + 1] = float(ratio[1]);
    float* terms = p.row_terms + p.rows;
    terms[i] = float(loss / count);
    terms[pairs + i] = float(double(p.beta) * ratio[0] / count);
    terms[2 * pairs + i] = float(double(p.beta) * ratio[1] / count);
    terms[3 * pairs + i] = ratio[0] > ratio[1] ? float(1.0 / count) : 0.0f;
    __threadfence();
    last = atomicAdd(&p.tickets[0], 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  double out[4];
  sum_columns<256>(p.row_terms + p.rows, pairs, pairs, 4, sums, out);
  if (threadIdx.x == 0)
    for (int c = 0; c < 4; ++c) p.stats[c] = float(out[c]);
}

// Launched so that it may be scheduled while the kernel before it drains; every
// kernel here waits for that one before it touches memory.
cudaError_t launch_after(void (*kernel)(LossParams), const LossParams& p, int64_t grid, int threads,
                         cudaStream_t stream) {
  if (grid <= 0) return cudaSuccess;
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(grid));
  cfg.blockDim = dim3(unsigned(threads));
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int MODE>
cudaError_t launch_rows(const LossParams& p, ar_dtype dtype, cudaStream_t stream) {
  return launch_after(dtype == AR_BF16 ? rows_kernel<true, MODE> : rows_kernel<false, MODE>, p, p.rows, kRowThreads,
                      stream);
}

}  // namespace

cudaError_t launch_token_logp(const LossParams& p, ar_dtype dtype, cudaStream_t stream) {
  return launch_rows<kLogp>(p, dtype, stream);
}

cudaError_t launch_policy_loss(const LossParams& p, ar_dtype dtype, cudaStream_t stream) {
  cudaError_t err = cudaMemsetAsync(p.tickets, 0, 8, stream);
  if (err == cudaSuccess && p.rows == 0) return cudaMemsetAsync(p.stats, 0, 16, stream);
  if (err == cudaSuccess) err = launch_after(count_kernel, p, p.n_seq, 256, stream);
  if (err == cudaSuccess) err = launch_rows<kPolicy>(p, dtype, stream);
  return err;
}

cudaError_t launch_preference_loss(const LossParams& p, ar_dtype dtype, cudaStream_t stream) {
  cudaError_t err = cudaMemsetAsync(p.tickets, 0, 8, stream);
  if (err == cudaSuccess) err = launch_rows<kPrefForward>(p, dtype, stream);
  if (err == cudaSuccess) err = launch_after(pair_kernel, p, p.n_seq / 2, 256, stream);
  if (err == cudaSuccess && p.d != nullptr) err = launch_rows<kPrefBackward>(p, dtype, stream);
  return err;
}

}  // namespace ar
