// Losses on a language model's logits, with their gradients: token
// log-probabilities, the clipped policy loss with a KL term, and the
// preference loss over paired log ratios.
//
// For row t with logits x, temperature tau and label y:
//   lp = x_y / tau - log sum_j exp(x_j / tau)
// and a loss that depends on the logits through lp alone has
//   dL/dx_j = (dL/dlp) * ([j = y] - p_j) / tau,   p_j = exp(x_j / tau) / sum.
//
// All of it is kept in base 2: with k = log2(e) / tau (rounded to fp32, which
// moves lp by at most 2^-24 (x_y - mean x) / tau, mean over p, alike in every call:
// differences of log-probabilities made here lose most of it) and any shift c,
// e_j = 2^(x_j k - c) is one FMA and one exponential, and two partial sums
// with shifts c1, c2 combine exactly by 2^(c1 - c2). Sums and shifts are fp32;
// the few operations a row does once (lp itself) are in pairs of fp32, so that
// lp carries no rounding of the shift or of the logarithm's integer part.
// Shifts are integers.
// Gradients are rounded once, into the logits' type.
//
// A row whose label is negative is not read: its log-probability is 0 and its
// gradient row is zeros, whatever the logits there hold. A label >= vocab
// makes its row NaN. A row of -inf alone has no distribution: NaN. A row of the
// type's lowest value alone is uniform.
//
// Kernels. All are bound by HBM where there are many rows (each unmasked row is
// read once, or twice for a preference loss, whose slopes need whole sequences
// first; each gradient row is written once), by launches and latency where
// there are few. One GB300, copy bandwidth 6771 GB/s:
//  stream_kernel  many long rows. 16384 x 32000 bf16, a quarter masked, policy
//                 loss: 298 us in the kernel for 1.77 GB, 0.88 of the copy
//                 bandwidth (two exponentials an element: special function
//                 unit 28 % busy, issue slots 51 %); 3001 x 32003 fp32: 112 us a call;
//                 log-probabilities of 6007 x 50021 bf16: 78 us, 0.86.
//  rows_kernel    a cluster of CTAs a row, the row in registers: 16 x 32000
//                 fp32 log-probabilities 4.0 us in a graph of calls
//  count_kernel, stats_kernel, pair_kernel  sequences; not needed where a call
//                 has a few rows (64-token policy loss 11 us in a graph of calls)
#include "loss.h"

#include <algorithm>
#include <array>
#include <mutex>
#include <vector>

#include "bulk.cuh"
#include "common.cuh"

namespace ar {
namespace {

// What one thread holds of a row: kVecs 16-byte vectors, so that a row is read
// once, its sum taken, and the gradient written from registers. With 512
// threads and clusters of up to 8 CTAs a row that is up to 8 x 32768 bf16 or
// 8 x 16384 fp32 long; longer ones are read twice.
constexpr int kVecs = 8;

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 operations an instruction.
struct Pair {
  uint64_t v;
};
__device__ __forceinline__ Pair pair_of(float lo, float hi) {
  Pair r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 floats_of(Pair a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
  Pair r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
// The pairs of a vector: 4 of bf16, 2 of fp32.
template <bool BF16>
__device__ __forceinline__ Pair pair_at(const uint4& r, int i) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
  if (BF16) return pair_of(bf16lo(w[i]), bf16hi(w[i]));
  return pair_of(__uint_as_float(w[2 * i % 4]), __uint_as_float(w[(2 * i + 1) % 4]));
}
// 2^(x k - shift) of both.
__device__ __forceinline__ Pair exp2_pair(Pair x, Pair k, Pair minus_shift) {
  const float2 y = floats_of(fma2(x, k, minus_shift));
  return pair_of(exp2_approx(y.x), exp2_approx(y.y));
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
// A join drops a part whose shift is 127 or more below the other's: sums have to
// be of the order of their number of terms, or normalized.
struct Lse {
  float c, s;
};
// The same value with its sum, a normal number, in [1/2, 1).
__device__ __forceinline__ Lse normalized(Lse v) {
  const int bits = __float_as_int(v.s);
  return {v.c + float((bits >> 23) - 126), __int_as_float((bits & 0x007fffff) | 0x3f000000)};
}
__device__ __forceinline__ Lse lse_join(Lse a, Lse b) {
  const float c = fmaxf(a.c, b.c), z = finite_shift(c);
  return {c, a.s * pow2(a.c - z) + b.s * pow2(b.c - z)};
}
__device__ __forceinline__ Lse lse_warp(Lse v, int width) {
  for (int o = width / 2; o > 0; o >>= 1)
    v = lse_join(v, {__shfl_xor_sync(~0u, v.c, o), __shfl_xor_sync(~0u, v.s, o)});
  return v;
}

// A warp's sum at the largest of its shifts: each part is scaled once.
__device__ __forceinline__ Lse lse_warp_at_max(Lse v) {
  float c;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(c) : "f"(v.c));
  float s = v.s * pow2(v.c - finite_shift(c));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
  return {c, s};
}

// A sum of two floats, for the few operations of a row that need more than 24 bits.
struct Two {
  float hi, lo;
};
__device__ __forceinline__ Two two_sum(float a, float b) {
  const float s = a + b, t = s - a;
  return {s, (a - (s - t)) + (b - t)};
}

// lp = (x_y k - c - log2 s) ln 2. What cancels is subtracted exactly.
__device__ __forceinline__ Two log_prob(float x, float k, Lse z) {
  // s = f * 2^e with f in [1/2, 1): the integer part of its logarithm is exact
  int e = 0;
  const float f = frexpf(z.s, &e), c = finite_shift(z.c);
  const float xk = x * k;
  const Two a = two_sum(xk, -c), b = two_sum(a.hi, -float(e)), d = two_sum(b.hi, -log2f(f));
  const float lo = fmaf(x, k, -xk) + a.lo + b.lo + d.lo;
  constexpr float kLn2 = 0.69314718f, kLn2Low = float(0.69314718055994530942 - double(kLn2));
  const float r = d.hi * kLn2;
  const float low = fmaf(d.hi, kLn2, -r) + fmaf(d.hi, kLn2Low, lo * kLn2);
  if (!isfinite(r) || low != low) return {r, 0.0f};  // -inf or NaN as it is
  return {r, low};
}

// The range of a row of `n` elements starting at `base`: `head` elements up to
// the first 16-byte boundary, `vecs` whole 16-byte vectors, the rest.
template <int W, int ES>
struct RowSpan {
  int head, vecs, tail;
  __device__ __forceinline__ RowSpan(const char* base, int n) {
    const int off = int(reinterpret_cast<uintptr_t>(base) % 16) / ES;
    head = off ? W - off : 0;
    if (head > n) head = n;
    vecs = (n - head) / W;
    tail = n - head - vecs * W;
  }
  // Which of `ranks` CTAs that share the row's vectors (see Slice) has element e; the first has what lies outside them.
  __device__ __forceinline__ int owner(int64_t e, int ranks) const {
    const int64_t at = e - head;
    return at < 0 || at >= int64_t(vecs) * W ? 0 : int(at) / W / ((vecs + ranks - 1) / ranks);
  }
  // The element outside the vectors that thread `i` takes (-1: none).
  __device__ __forceinline__ int edge(int i) const {
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

// A vector of the logits' type (bf16: two conversions an instruction).
__device__ __forceinline__ uint4 narrow(const float (&f)[4]) { return Lane<false, true>::narrow(f); }
__device__ __forceinline__ uint4 narrow(const float (&f)[8]) {
  uint4 r;
  auto two = [](float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  };
  r.x = two(f[0], f[1]), r.y = two(f[2], f[3]), r.z = two(f[4], f[5]), r.w = two(f[6], f[7]);
  return r;
}

// The part of a row that one CTA of its cluster takes.
template <bool BF16, int THREADS>
struct Slice {
  static constexpr int W = Lane<BF16, true>::W, ES = BF16 ? 2 : 4;
  static constexpr int kChunk = THREADS * kVecs;  // vectors held at a time
  const char* x;
  RowSpan<W, ES> span;
  int v0, v1;
  int edge;  // this thread's element outside the vectors, -1: none
  __device__ __forceinline__ Slice(const char* row, int vocab, int rank, int ranks) : x(row), span(row, vocab) {
    const int per = (span.vecs + ranks - 1) / ranks;
    v0 = min(span.vecs, per * rank);
    v1 = min(span.vecs, v0 + per);
    edge = rank == 0 ? span.edge(threadIdx.x) : -1;
  }
  __device__ __forceinline__ bool held() const { return v1 - v0 <= kChunk; }
  // Vectors first + threadIdx.x + j THREADS, -inf beyond the slice.
  __device__ __forceinline__ void load(uint4 (&raw)[kVecs], int first) const {
    const uint32_t none = BF16 ? 0xFF80FF80u : 0xFF800000u;
    const int v = first + int(threadIdx.x);
    const uint4* from = reinterpret_cast<const uint4*>(x + span.head * ES) + v;
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      raw[j] = make_uint4(none, none, none, none);
      if (v + j * THREADS < v1) raw[j] = __ldcs(from + j * THREADS);
    }
  }
};

// (The packed bf16 maximum instruction measured 1.6 times slower over a whole
// row than widening first.)
template <bool BF16>
__device__ __forceinline__ float largest(const uint4& r) {
  constexpr int W = Lane<BF16, true>::W;
  float f[W];
  Lane<BF16, true>::widen(r, f);
  float m = f[0];
#pragma unroll
  for (int w = 1; w < W; ++w) m = fmaxf(m, f[w]);
  return m;
}

// This thread's share of the row's sum.
template <bool BF16>
__device__ __forceinline__ Lse thread_lse(const uint4 (&raw)[kVecs], float k) {
  constexpr int W = Lane<BF16, true>::W;
  float top = largest<BF16>(raw[0]);
#pragma unroll
  for (int j = 1; j < kVecs; ++j) top = fmaxf(top, largest<BF16>(raw[j]));
  const float c = fmaxf(-INFINITY, ceilf(top * k)), shift = finite_shift(c);  // (fmaxf: a NaN alone)
  float s[2] = {0.0f, 0.0f};
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    float f[W];
    Lane<BF16, true>::widen(raw[j], f);
#pragma unroll
    for (int w = 0; w < W; ++w) s[w & 1] += exp2_approx(fmaf(f[w], k, -shift));
  }
  return {c, s[0] + s[1]};
}

// (RUNS: nothing but that this thread's CTA runs is told, and no fence taken)
template <bool RUNS = false>
__device__ __forceinline__ void cluster_arrive() {
  if (RUNS) asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
  else asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ void cluster_barrier() {
  cluster_arrive();
  cluster_wait();
}
__device__ __forceinline__ void store_peer(void* p, int rank, float2 v) {
  const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p));
  asm volatile(
      "{\n"
      ".reg .b32 remote;\n"
      "mapa.shared::cluster.u32 remote, %0, %1;\n"
      "st.shared::cluster.v2.f32 [remote], {%2, %3};\n"
      "}\n" ::"r"(a),
      "r"(rank), "f"(v.x), "f"(v.y)
      : "memory");
}

// The same counted (16 bytes) on a barrier of that CTA, which needs no fence between the CTAs.
__device__ __forceinline__ void send_peer(void* p, uint64_t* bar, int rank, float4 v) {
  asm volatile(
      "{\n"
      ".reg .b32 to, count;\n"
      "mapa.shared::cluster.u32 to, %0, %2;\n"
      "mapa.shared::cluster.u32 count, %1, %2;\n"
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [to], {%3, %4, %5, %6}, [count];\n"
      "}\n" ::"r"(smem_u32(p)),
      "r"(smem_u32(bar)), "r"(rank), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
      : "memory");
}

// One token's part of the policy loss.
struct PolicyTerm {
  float terms[3];  // weighted surrogate, KL, whether the clip holds the ratio
  float up;        // slope of the loss in x_y
};
__device__ __forceinline__ PolicyTerm policy_term(const LossParams& p, float lp, float weight, float mean, float adv,
                                                  float old, float ref) {
  const float ratio = expf(lp - old);
  const float free = adv == 0.0f && ratio == INFINITY ? 0.0f : ratio * adv;  // (beyond fp32's range, not infinite)
  const float held = (ratio < p.lo ? p.lo : ratio > p.hi ? p.hi : ratio) * adv;  // NaN stays NaN
  const float w = weight * mean;
  float slope = free <= held ? -free : free > held ? 0.0f : free;
  PolicyTerm r = {{-w * (free < held || free != free ? free : held), 0.0f, held < free ? w : 0.0f}, 0.0f};
  if (p.ref_logp != nullptr) {
    const float back = ref - lp, grow = expm1f(back);
    r.terms[1] = w * (grow == INFINITY ? grow : grow - back);
    if (p.kl > 0.0f) slope -= p.kl * grow;  // (a coefficient of 0: no part of the loss, infinite or not)
  }
  r.up = w * slope * p.grad_scale * p.inv_temp;
  if (weight == 0.0f) r = {{0.0f, 0.0f, 0.0f}, 0.0f};  // outside every sequence
  return r;
}

constexpr int kMaxCluster = 8;
struct RowShared {
  Lse warp[16];
  float2 cta[kMaxCluster];
};

// The row's sum, from every thread's; the same bits in every thread of the
// cluster. Every thread has arrived at the cluster's barrier before: only when
// all have (the peers run, and are done with an earlier sum) is a peer's shared
// memory written to.
template <int THREADS>
__device__ __forceinline__ Lse row_sum(Lse v, RowShared& sh, int rank, int ranks) {
  constexpr int W = THREADS / 32;
  v = lse_warp(v, 32);
  if (threadIdx.x % 32 == 0) sh.warp[threadIdx.x / 32] = v;
  __syncthreads();
  v = lse_warp(sh.warp[threadIdx.x % W], W);
  if (ranks > 1) {
    cluster_wait();
    if (threadIdx.x < ranks) store_peer(&sh.cta[rank], threadIdx.x, make_float2(v.c, v.s));
    cluster_barrier();
    v = {sh.cta[0].x, sh.cta[0].y};
    for (int r = 1; r < ranks; ++r) v = lse_join(v, {sh.cta[r].x, sh.cta[r].y});
  }
  return v;
}

template <bool BF16, int THREADS>
__device__ __forceinline__ Lse row_lse(const Slice<BF16, THREADS>& slice, uint4 (&raw)[kVecs], float edge, float k,
                                       RowShared& sh, int rank, int ranks) {
  Lse z = {-INFINITY, 0.0f};
  if (slice.held()) {
    z = thread_lse<BF16>(raw, k);
  } else {
#pragma unroll 1
    for (int first = slice.v0; first < slice.v1; first += slice.kChunk) {
      slice.load(raw, first);
      z = lse_join(z, thread_lse<BF16>(raw, k));
    }
  }
  if (slice.edge >= 0) {
    const float c = fmaxf(-INFINITY, ceilf(edge * k));
    z = lse_join(z, {c, exp2_approx(fmaf(edge, k, -finite_shift(c)))});
  }
  return row_sum<THREADS>(z, sh, rank, ranks);
}

// The gradient of this CTA's part of a row, from the vectors held:
// d_j = up * [j = y] - up * p_j, p_j = 2^(x_j k - shift) * inv_sum.
template <bool BF16, int THREADS>
__device__ __forceinline__ void write_gradient(const Slice<BF16, THREADS>& slice, char* d, uint4 (&raw)[kVecs], float edge,
                                               int64_t label, float up, float k, float shift, float inv_sum) {
  using L = Lane<BF16, true>;
  constexpr int W = L::W;
  const bool aligned = (reinterpret_cast<uintptr_t>(d) - reinterpret_cast<uintptr_t>(slice.x)) % 16 == 0;
  const float g = -up * inv_sum;
  const int own = int(label) - slice.span.head;  // the label's place among the vectors' elements
#pragma unroll 1
  for (int first = slice.v0; first < slice.v1; first += slice.kChunk) {
    if (!slice.held()) slice.load(raw, first);
    const int v = first + int(threadIdx.x);
    char* to = d + (slice.span.head + int64_t(v) * W) * slice.ES;
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      if (v + j * THREADS >= slice.v1) continue;
      float f[W];
      L::widen(raw[j], f);
#pragma unroll
      for (int w = 0; w < W; ++w) f[w] = exp2_approx(fmaf(f[w], k, -shift)) * g;
      const int at = own - (v + j * THREADS) * W;
      if (unsigned(at) < unsigned(W)) {
#pragma unroll
        for (int w = 0; w < W; ++w)
          if (at == w) f[w] += up;
      }
      if (aligned) {
        L::store(to, j * THREADS * W, narrow(f));
      } else {
#pragma unroll
        for (int w = 0; w < W; ++w) store_one<BF16>(to, j * THREADS * W + w, f[w]);
      }
    }
  }
  if (slice.edge >= 0) {
    const float v = exp2_approx(fmaf(edge, k, -shift)) * g;
    store_one<BF16>(d, slice.edge, label == slice.edge ? v + up : v);
  }
}

// Zeros in this CTA's part of a gradient row.
template <bool BF16, int THREADS>
__device__ __forceinline__ void write_zeros(char* d, int vocab, int rank, int ranks) {
  const Slice<BF16, THREADS> slice(d, vocab, rank, ranks);
  uint4* to = reinterpret_cast<uint4*>(d + slice.span.head * slice.ES);
  for (int v = slice.v0 + int(threadIdx.x); v < slice.v1; v += THREADS) __stcs(to + v, make_uint4(0, 0, 0, 0));
  if (slice.edge >= 0) store_one<BF16>(d, slice.edge, 0.0f);
}

// ---------------------------------------------------------------- sequences

__device__ __forceinline__ int64_t seq_bound(const LossParams& p, int64_t i) {
  const int64_t v = p.seq_start == nullptr ? (i == 0 ? 0 : p.rows) : p.seq_start[i];
  return v < 0 ? int64_t(0) : v > p.rows ? p.rows : v;
}

// Labelled tokens of each sequence (one CTA a sequence), and the rows' weights
// before the mean's denominator.
__global__ void __launch_bounds__(256) count_kernel(LossParams p) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t s = blockIdx.x, lo = seq_bound(p, s), hi = seq_bound(p, s + 1);
  __shared__ int warp_sum[8];
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
  if (threadIdx.x == 0) p.seq_count[s] = n;
}

// 1 / (the mean's denominator), by one warp.
__device__ __forceinline__ float mean_scale(const LossParams& p) {
  if (p.denominator > 0.0f) return 1.0f / p.denominator;
  int64_t sum = 0;
  for (int64_t i = threadIdx.x % 32; i < p.n_seq; i += 32) {
    const int c = p.seq_count[i];
    sum += p.by_sequence ? (c > 0) : c;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
  return 1.0f / float(sum > 0 ? sum : 1);
}

// Sums `n` entries of each of COLUMNS columns (`pitch` apart) in a fixed order,
// by the CTA; results in thread 0.
template <int THREADS, int COLUMNS>
__device__ __forceinline__ void sum_columns(const float* col, int64_t pitch, int64_t n, float (&out)[COLUMNS]) {
  __shared__ float warp_sum[COLUMNS][THREADS / 32];
  float a[COLUMNS] = {};
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < n; i += THREADS)
#pragma unroll
    for (int c = 0; c < COLUMNS; ++c) a[c] += __ldcg(col + c * pitch + i);
#pragma unroll
  for (int c = 0; c < COLUMNS; ++c) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a[c] += __shfl_xor_sync(~0u, a[c], o);
    if (threadIdx.x % 32 == 0) warp_sum[c][threadIdx.x / 32] = a[c];
  }
  __syncthreads();
#pragma unroll
  for (int c = 0; c < COLUMNS; ++c) {
    out[c] = 0.0f;
    if (threadIdx.x == 0)
      for (int w = 0; w < THREADS / 32; ++w) out[c] += warp_sum[c][w];
  }
}

// Calls of a few rows do without the kernels that count sequences and join
// pairs: every CTA of the rows' kernels does that for its own row, while its
// part of the row is on the way.
constexpr int kFewRows = 512, kFewSequences = 32;

struct FewShared {
  int64_t bound[kFewSequences + 1];
  int count[kFewSequences];
};

// Bounds of the sequences (shared memory), and the one that row t is in (-1:
// none). Ends with the bounds visible to the CTA.
template <int THREADS>
__device__ __forceinline__ void few_bounds(const LossParams& p, FewShared& sh) {
  if (threadIdx.x <= p.n_seq) sh.bound[threadIdx.x] = seq_bound(p, threadIdx.x);
  if (threadIdx.x < p.n_seq) sh.count[threadIdx.x] = 0;
  __syncthreads();
}
__device__ __forceinline__ int few_sequence(const LossParams& p, const FewShared& sh, int64_t t) {
  for (int s = 0; s < p.n_seq; ++s)
    if (t >= sh.bound[s] && t < sh.bound[s + 1]) return s;
  return -1;
}

// A row's weight, the mean's denominator included.
template <int THREADS>
__device__ __forceinline__ float few_weight(const LossParams& p, FewShared& sh, int64_t t) {
  few_bounds<THREADS>(p, sh);
  for (int64_t r = threadIdx.x; r < p.rows; r += THREADS)
    if (p.labels[r] >= 0) {
      const int s = few_sequence(p, sh, r);
      if (s >= 0) atomicAdd(&sh.count[s], 1);
    }
  __syncthreads();
  int total = 0;
  for (int s = 0; s < p.n_seq; ++s) total += p.by_sequence ? sh.count[s] > 0 : sh.count[s];
  const int own = few_sequence(p, sh, t);
  if (own < 0) return 0.0f;
  const float weight = p.by_sequence ? 1.0f / float(max(sh.count[own], 1)) : 1.0f;
  return weight * (p.denominator > 0.0f ? 1.0f / p.denominator : 1.0f / float(max(total, 1)));
}

// The log ratio of a sequence before any division, and its labelled tokens, by one warp.
__device__ __forceinline__ Two add_two(Two a, float hi, float lo) {
  const Two s = two_sum(a.hi, hi);
  return {s.hi, a.lo + s.lo + lo};
}
__device__ __forceinline__ Two warp_ratio(const LossParams& p, int64_t lo, int64_t hi, int& count) {
  Two a = {0.0f, 0.0f};
  int n = 0;
#pragma unroll 4
  for (int64_t t = lo + threadIdx.x % 32; t < hi; t += 32)
    if (p.labels[t] >= 0) {
      a = add_two(a, __ldcg(&p.row_terms[t]), 0.0f);
      ++n;
    }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a = add_two(a, __shfl_xor_sync(~0u, a.hi, o), __shfl_xor_sync(~0u, a.lo, o));
  count = __reduce_add_sync(~0u, n);
  return a;
}

// One pair: statistics' terms and the coefficients of its rows.
struct PairTerms {
  float ratio[2], terms[4], coef[2];
};
__device__ __forceinline__ PairTerms pair_terms(const LossParams& p, const Two (&sum)[2], const int (&n)[2]) {
  PairTerms r;
  const float count = p.denominator > 0.0f ? p.denominator : float(p.n_seq / 2);
  float over[2];
  for (int h = 0; h < 2; ++h) {
    over[h] = p.normalize ? float(max(n[h], 1)) : 1.0f;
    r.ratio[h] = (sum[h].hi + sum[h].lo) / over[h];
    if (!isfinite(r.ratio[h])) r.ratio[h] = sum[h].hi;  // (an infinity has no low part)
  }
  // without the length, the difference of the ratios comes before their rounding
  const float apart = p.normalize || !isfinite(r.ratio[0] - r.ratio[1])
                          ? r.ratio[0] - r.ratio[1]
                          : (sum[0].hi - sum[1].hi) + (sum[0].lo - sum[1].lo);
  const float z = p.beta * apart;
  float loss, slope;
  if (p.square) {
    const float off = z - p.target;
    loss = off * off;
    slope = 2.0f * off;
  } else {
    // log1p(e^-|z|) serves both signs of z
    const float tail = log1pf(expf(-fabsf(z))), up = z > 0.0f ? z : 0.0f, down = z < 0.0f ? -z : 0.0f;
    loss = (1.0f - p.smooth) * (tail + down);
    if (p.smooth > 0.0f) loss += p.smooth * (tail + up);  // (up may be infinite)
    slope = -(1.0f - p.smooth) / (1.0f + expf(z)) + p.smooth / (1.0f + expf(-z));
    if (z != z) loss = slope = z;
  }
  for (int h = 0; h < 2; ++h)
    r.coef[h] = (h ? -1.0f : 1.0f) * slope * p.beta / count / over[h] * p.grad_scale;
  r.terms[0] = loss / count;
  r.terms[1] = p.beta * r.ratio[0] / count;
  r.terms[2] = p.beta * r.ratio[1] / count;
  r.terms[3] = r.ratio[0] > r.ratio[1] ? 1.0f / count : 0.0f;
  return r;
}

// The coefficient of row t; the first CTA also writes ratios and statistics.
template <int THREADS>
__device__ __forceinline__ float few_coefficient(const LossParams& p, FewShared& sh, int64_t t, bool first) {
  __shared__ Two sum[kFewSequences];
  __shared__ float terms[4][kFewSequences / 2];
  few_bounds<THREADS>(p, sh);
  const int warp = threadIdx.x / 32, own = few_sequence(p, sh, t);
  // the row's pair, or all of them
  const int from = first ? 0 : own < 0 ? 0 : own / 2 * 2, to = first ? int(p.n_seq) : own < 0 ? 0 : from + 2;
  for (int s = from + warp; s < to; s += THREADS / 32) {
    int n;
    const Two a = warp_ratio(p, sh.bound[s], sh.bound[s + 1], n);
    if (threadIdx.x % 32 == 0) {
      sum[s] = a;
      sh.count[s] = n;
    }
  }
  __syncthreads();
  auto pair = [&](int i) {
    const Two two[2] = {sum[2 * i], sum[2 * i + 1]};
    const int n[2] = {sh.count[2 * i], sh.count[2 * i + 1]};
    return pair_terms(p, two, n);
  };
  if (first) {
    const int i = threadIdx.x;
    if (i < p.n_seq / 2) {
      const PairTerms r = pair(i);
      p.ratios[2 * i] = r.ratio[0];
      p.ratios[2 * i + 1] = r.ratio[1];
      for (int c = 0; c < 4; ++c) terms[c][i] = r.terms[c];
    }
    __syncthreads();
    if (threadIdx.x < 4) {
      float a = 0.0f;
      for (int k = 0; k < p.n_seq / 2; ++k) a += terms[threadIdx.x][k];
      p.stats[threadIdx.x] = a;
    }
  }
  return own < 0 ? 0.0f : pair(own / 2).coef[own & 1];
}

// ---------------------------------------------------------------- rows

// One cluster a row.
template <bool BF16, int MODE, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) rows_kernel(LossParams p) {
  constexpr int ES = BF16 ? 2 : 4;
  __shared__ RowShared sh;
  __shared__ float mean_shared;
  grid_dependency_wait();
  grid_dependents_launch();
  const int ranks = p.cluster, rank = int(blockIdx.x) % ranks;
  const int64_t t = blockIdx.x / ranks;
  const char* x = static_cast<const char*>(p.x) + t * p.ld * ES;
  char* d = p.d == nullptr ? nullptr : static_cast<char*>(p.d) + t * p.dld * ES;
  if (MODE == kPrefForward && blockIdx.x == 0 && threadIdx.x == 0) p.tickets[0] = 0;
  const int64_t label = p.labels[t];
  __shared__ FewShared few;
  const bool first = blockIdx.x == 0;
  if (label < 0) {
    if (MODE == kPrefBackward && p.few && first) few_coefficient<THREADS>(p, few, t, true);
    if ((MODE == kPolicy || MODE == kPrefBackward) && d != nullptr) write_zeros<BF16, THREADS>(d, int(p.vocab), rank, ranks);
    if (MODE != kPrefBackward && rank == 0 && threadIdx.x == 0) {
      p.logp[t] = 0.0f;
      if (MODE == kPolicy)
        for (int c = 0; c < 3; ++c) p.row_terms[c * p.rows + t] = 0.0f;
    }
    return;
  }
  // (all CTAs of a cluster have the same row: they return above together, or come here)
  if (MODE != kPrefBackward && ranks > 1) cluster_arrive<true>();  // waited for in row_sum, behind the loads
  const Slice<BF16, THREADS> slice(x, int(p.vocab), rank, ranks);
  uint4 raw[kVecs];
  slice.load(raw, slice.v0);
  const float edge = slice.edge >= 0 ? load_one<BF16>(x, slice.edge) : -INFINITY;
  if (MODE == kPrefBackward) {
    const float2 z = p.row_lse[t];  // the sign of 1 / sum tells the scale
    const float coef = p.few ? few_coefficient<THREADS>(p, few, t, first) : p.row_a[t];
    if (coef == 0.0f) {  // outside every sequence, mostly: zeros, whatever the row holds
      write_zeros<BF16, THREADS>(d, int(p.vocab), rank, ranks);
      return;
    }
    write_gradient<BF16, THREADS>(slice, d, raw, edge, label, coef * p.inv_temp, z.y < 0.0f ? 1.0f : p.k, z.x,
                                  fabsf(z.y));
    return;
  }
  const float nan = __int_as_float(0x7fffffff);
  // (barriers follow: this is read before any gradient is written)
  const float x_label = label < p.vocab ? load_one<BF16>(x, label) : nan;
  float weight = 0.0f, adv = 0.0f, old = 0.0f, ref = 0.0f;
  if (MODE == kPolicy) {
    adv = p.adv[t];
    old = p.old_logp[t];
    if (p.few) {
      weight = few_weight<THREADS>(p, few, t);
    } else {
      weight = p.row_a[t];
      if (threadIdx.x < 32) {
        const float m = mean_scale(p);
        if (threadIdx.x == 0) mean_shared = m;
      }
    }
  }
  if ((MODE == kPolicy || MODE == kPrefForward) && p.ref_logp != nullptr) ref = p.ref_logp[t];
  // Where x k itself is not finite (a row whose largest logit is near the
  // type's lowest or highest value), two logits differ by 0 or by more than any
  // exponent holds, at any scale: k = 1 serves.
  float k = p.k;
  Lse z = row_lse<BF16, THREADS>(slice, raw, edge, k, sh, rank, ranks);
  if (isinf(z.c)) {
    k = 1.0f;
    __syncthreads();
    if (ranks > 1) cluster_arrive();
    z = row_lse<BF16, THREADS>(slice, raw, edge, k, sh, rank, ranks);
  }
  const Two exact = log_prob(x_label, k, z);
  const float lp = exact.hi + exact.lo, shift = finite_shift(z.c), inv_sum = 1.0f / z.s;
  const bool teller = rank == 0 && threadIdx.x == 0;
  if (teller) p.logp[t] = lp;
  if (MODE == kPrefForward && teller) {
    // the log ratio before lp is rounded: sequences sum hundreds of them
    p.row_terms[t] = (exact.hi - ref) + exact.lo;
    p.row_lse[t] = make_float2(shift, copysignf(inv_sum, k == p.k ? 1.0f : -1.0f));
  }
  if (MODE != kPolicy) return;
  const PolicyTerm term = policy_term(p, lp, weight, p.few ? 1.0f : mean_shared, adv, old, ref);
  if (d != nullptr) {
    if (weight == 0.0f)
      write_zeros<BF16, THREADS>(d, int(p.vocab), rank, ranks);
    else
      write_gradient<BF16, THREADS>(slice, d, raw, edge, label, label < p.vocab ? term.up : nan, k, shift, inv_sum);
  }
  if (teller)
    for (int c = 0; c < 3; ++c) p.row_terms[c * p.rows + t] = term.terms[c];
}

// ---------------------------------------------------------------- many rows

// Rows streamed through shared memory, for calls with many long rows: one
// persistent CTA an SM, clusters of `p.cluster` CTAs sharing each row. A
// producer warp copies rows in chunks of 32 KB, up to three rows ahead; 16
// warps take sums and write gradients; one warp finishes a row (joins the
// warps' and the cluster's sums, takes the logarithm, decides the loss's slope).
// The sums of row n + 1 are taken before the gradient of row n is written, from
// the same shared memory, so nothing waits for the finisher and each row
// crosses HBM once each way.
constexpr int kStreamWarps = 16, kStreamThreads = kStreamWarps * 32 + 64;
constexpr int kStreamChunk = 32768, kStreamChunks = 6, kStreamRows = 4;
constexpr int kStreamSlice = 65536;  // bytes of a row per CTA, at most, where a row is held until its gradient is written
constexpr uint32_t kWaitPolls = 1u << 22;

struct StreamRow {
  int64_t t, label;   // t < 0: no more rows
  int head, v0, v1;   // elements before the vectors; this CTA's vectors
};
struct StreamResult {
  float k, shift, g, up;
  int zeros;  // the gradient is zeros, whatever the row holds
};
struct StreamShared {
  uint64_t full[kStreamChunks], empty[kStreamChunks];
  uint64_t row_full[kStreamRows], row_free[kStreamRows], sum_full[kStreamRows], result_full[kStreamRows];
  uint64_t cta_full[kStreamRows];
  StreamRow row[kStreamRows];
  StreamResult result[kStreamRows];
  Lse warp_sum[kStreamRows][kStreamWarps];
  float4 cta_sum[kStreamRows][kMaxCluster];  // shift, sum, the label's logit where the CTA has it
  int abort_flag;
};

// A copy of what is not read again soon. (Keeping the last 40 to 110 MB of the
// logits in the L2 between a pair's two passes changed nothing: 227 to 229 us.)
__device__ __forceinline__ void stream_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar,
                                            uint64_t evict_first) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar)), "l"(evict_first)
      : "memory");
}

// Adds a vector to a running sum, raising its shift where needed.
template <bool BF16>
__device__ __forceinline__ void lse_add(Lse& z, const uint4& raw, float k) {
  constexpr int W = Lane<BF16, true>::W;
  const float c = ceilf(largest<BF16>(raw) * k);
  if (c > z.c) {
    z.s *= pow2(z.c - c);
    z.c = c;
  }
  const float shift = finite_shift(z.c);
  float f[W];
  Lane<BF16, true>::widen(raw, f);
#pragma unroll
  for (int w = 0; w < W; ++w) z.s += exp2_approx(fmaf(f[w], k, -shift));
}

// The terms of a vector at a fixed shift.
template <bool BF16>
__device__ __forceinline__ Pair terms_of(const uint4& raw, Pair k, Pair minus_shift) {
  constexpr int P = Lane<BF16, true>::W / 2;
  Pair f[P];
#pragma unroll
  for (int w = 0; w < P; ++w) f[w] = exp2_pair(pair_at<BF16>(raw, w), k, minus_shift);
#pragma unroll
  for (int n = P / 2; n > 0; n /= 2)
#pragma unroll
    for (int w = 0; w < n; ++w) f[w] = add2(f[w], f[w + n]);
  return f[0];
}

// A vector of the gradient but for the label's element: 2^(x k - shift) g.
template <bool BF16>
__device__ __forceinline__ void gradient_of(const uint4& raw, Pair k, Pair minus_shift, Pair g,
                                            float (&f)[Lane<BF16, true>::W]) {
#pragma unroll
  for (int w = 0; w < Lane<BF16, true>::W / 2; ++w) {
    const float2 y = floats_of(mul2(exp2_pair(pair_at<BF16>(raw, w), k, minus_shift), g));
    f[2 * w] = y.x;
    f[2 * w + 1] = y.y;
  }
}

// A thread of the streaming kernel takes its shift from the first vectors of a
// row that it sees, and no maximum after that: fp32 holds terms up to 2^127
// times the shift's. Where those vectors are ruled out, kLeastShift serves. A
// sum that does not fit (an overflow; logits too low for kLeastShift) is taken
// again by its thread, from memory, with the maximum. What kLeastShift turns
// into 0 altogether is below 2^kLeastPart, in all of a row's threads: it counts
// for nothing beside a part above that, and else the finisher sums the row again.
// (Left to the finisher, one warp a row, every overflow made 6007 x 50021 bf16 at
// temperature 0.01 take 4.2 ms; taken again by the threads 0.38 ms, 0.09 without.)
constexpr float kLeastShift = -64.0f, kLeastPart = -140.0f;

template <bool BF16, int MODE>
__global__ void __launch_bounds__(kStreamThreads, 1) stream_kernel(LossParams p) {
  using L = Lane<BF16, true>;
  constexpr int W = L::W, ES = BF16 ? 2 : 4;
  constexpr bool SUM = MODE != kPrefBackward, WRITE = MODE == kPolicy || MODE == kPrefBackward;
  constexpr int kVecsChunk = kStreamChunk / 16, kThreadVecs = kVecsChunk / (kStreamWarps * 32);
  using Part = Slice<BF16, kStreamWarps * 32>;
  extern __shared__ char raw_shared[];
  char* chunks = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(raw_shared) + 127) & ~uintptr_t(127));
  __shared__ StreamShared sh;
  volatile int* abort = &sh.abort_flag;
  const StatusRef status = {p.status_word, p.status_host};
  const int ranks = p.cluster, rank = int(blockIdx.x) % ranks;
  const int64_t worker = blockIdx.x / ranks, workers = gridDim.x / ranks;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStreamChunks; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], kStreamWarps);
    }
    for (int i = 0; i < kStreamRows; ++i) {
      mbar_init(&sh.row_full[i], 1);
      mbar_init(&sh.row_free[i], kStreamWarps + 1);
      mbar_init(&sh.sum_full[i], kStreamWarps);
      mbar_init(&sh.result_full[i], 1);
      mbar_init(&sh.cta_full[i], 1);
    }
    sh.abort_flag = 0;
    mbar_init_fence();
  }
  __syncthreads();
  if (ranks > 1) cluster_barrier();
  grid_dependency_wait();
  grid_dependents_launch();
  if (MODE == kPrefForward && blockIdx.x == 0 && threadIdx.x == 0) p.tickets[0] = 0;
  auto row_of = [&](int64_t t) { return static_cast<const char*>(p.x) + t * p.ld * ES; };
  auto wait = [&](uint64_t* bar, int n, int ring) {
    return mbar_wait(&bar[n % ring], (n / ring) & 1, kWaitPolls, abort, status);
  };

  if (warp == kStreamWarps) {
    // ---- producer
    if (lane == 0) {
      uint64_t evict_first;
      asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(evict_first));
      int chunk = 0;
      // A preference loss's second pass goes backwards, from the rows that the
      // first one read last: 8192 x 32000 bf16 230.6 us a call and 233.4
      // forwards, 3500 x 131072 365 and 368.
      auto row_at = [&](int64_t i) { return MODE == kPrefBackward ? p.rows - 1 - i : i; };
      int64_t ahead = worker < p.rows ? p.labels[row_at(worker)] : -1;
      // Tells the others of the n-th row. Row n + 1 is told of before row n is
      // copied: the finisher looks it up before it finishes row n, and a row
      // may be longer than the ring.
      auto announce = [&](int n, StreamRow& r) {
        const int64_t i = worker + n * workers;
        r = {-1, ahead, 0, 0, 0};
        if (i < p.rows) {
          r.t = row_at(i);
          // a masked row's gradient is written at its own alignment
          const char* at = ahead < 0 && WRITE && p.d != nullptr ? static_cast<const char*>(p.d) + r.t * p.dld * ES : row_of(r.t);
          const Part part(at, int(p.vocab), rank, ranks);
          r.head = part.span.head, r.v0 = part.v0, r.v1 = part.v1;
        }
        if (i + workers < p.rows) ahead = p.labels[row_at(i + workers)];
        if (n >= kStreamRows && !wait(sh.row_free, n - kStreamRows, kStreamRows)) return false;
        sh.row[n % kStreamRows] = r;
        mbar_arrive(&sh.row_full[n % kStreamRows]);
        return true;
      };
      StreamRow r, after;
      bool more = announce(0, r);
      for (int n = 0; more && r.t >= 0 && !*abort; ++n, r = after) {
        more = announce(n + 1, after);
        if (r.label < 0) continue;
        const char* from = row_of(r.t) + r.head * ES;
        for (int v = r.v0; v < r.v1; v += kVecsChunk, ++chunk) {
          if (chunk >= kStreamChunks && !wait(sh.empty, chunk - kStreamChunks, kStreamChunks)) break;
          const uint32_t bytes = uint32_t(min(r.v1 - v, kVecsChunk)) * 16;
          mbar_arrive_expect_tx(&sh.full[chunk % kStreamChunks], bytes);
          stream_load(chunks + chunk % kStreamChunks * kStreamChunk, from + int64_t(v) * 16, bytes,
                      &sh.full[chunk % kStreamChunks], evict_first);
        }
      }
      // copies in flight land before the shared memory goes away
      for (int j = max(0, chunk - kStreamChunks); j < chunk; ++j)
        for (uint32_t k = 0; k < kWaitPolls && !mbar_try_wait(&sh.full[j % kStreamChunks], (j / kStreamChunks) & 1); ++k) {
        }
    }
  } else if (warp < kStreamWarps) {
    // ---- sums and gradients
    const int tid = threadIdx.x;
    constexpr int kStep = kStreamWarps * 32;
    int summed = 0, written = 0;  // ring places of the next chunk
    uint32_t sum_phase = 0, write_phase = 0;
    auto advance = [](int& at, uint32_t& phase) {
      if (++at == kStreamChunks) {
        at = 0;
        phase ^= 1;
      }
    };
    auto sum_row = [&](int n, const StreamRow& r) {
      Lse z = {-INFINITY, 0.0f};
      if (r.label >= 0) {
        const Pair kk = pair_of(p.k, p.k);
        Pair ss = pair_of(0.0f, 0.0f), sum = ss;
#pragma unroll 1
        for (int v = r.v0; v < r.v1; v += kVecsChunk) {
          if (!mbar_wait(&sh.full[summed], sum_phase, kWaitPolls, abort, status)) return false;
          const uint4* in = reinterpret_cast<const uint4*>(chunks + summed * kStreamChunk) + tid;
          const int left = r.v1 - v - tid;  // vectors from this thread's first one on
          uint4 raw[kThreadVecs];
#pragma unroll
          for (int j = 0; j < kThreadVecs; ++j)
            if (j * kStep < left) raw[j] = in[j * kStep];
          if (v == r.v0 && left > 0) {
            float top = largest<BF16>(raw[0]);
            if (kStep < left) top = fmaxf(top, largest<BF16>(raw[1]));
            z.c = fmaxf(-INFINITY, ceilf(top * p.k));  // (fmaxf: a NaN alone)
            if (z.c == -INFINITY) z.c = kLeastShift;
            ss = pair_of(-z.c, -z.c);
          }
#pragma unroll
          for (int j = 0; j < kThreadVecs; ++j)
            if (j * kStep < left) sum = add2(sum, terms_of<BF16>(raw[j], kk, ss));
          if (!WRITE) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.empty[summed]);
          }
          advance(summed, sum_phase);
        }
        const float2 both = floats_of(sum);
        z.s = both.x + both.y;
        if (!(z.s < INFINITY) || (z.c == kLeastShift && z.s > 0.0f && z.s < 0x1p-60f)) {
          z = {-INFINITY, 0.0f};
          const uint4* in = reinterpret_cast<const uint4*>(row_of(r.t) + r.head * ES);
          for (int v = r.v0 + tid; v < r.v1; v += kStep) lse_add<BF16>(z, in[v], p.k);
        }
        if (z.s > 0.0f && z.s < INFINITY) z = normalized(z);
        else if (z.c == kLeastShift) z.c = kLeastPart;
        z = lse_warp_at_max(z);
      }
      if (lane == 0) {
        sh.warp_sum[n % kStreamRows][warp] = z;
        mbar_arrive(&sh.sum_full[n % kStreamRows]);
      }
      return true;
    };
    auto write_row = [&](int n, const StreamRow& r) {
      if (!wait(sh.result_full, n, kStreamRows)) return false;
      const StreamResult q = sh.result[n % kStreamRows];
      char* d = static_cast<char*>(p.d) + r.t * p.dld * ES + r.head * ES;
      if (r.label < 0) {
        if (p.d != nullptr)
          for (int v = r.v0 + tid; v < r.v1; v += kStep) __stcs(reinterpret_cast<uint4*>(d) + v, make_uint4(0, 0, 0, 0));
        return true;
      }
      const bool aligned = reinterpret_cast<uintptr_t>(d) % 16 == 0;
      if (q.zeros) {  // the row's chunks are passed over (with a test at each vector instead, a call took 3 % longer)
        for (int v = r.v0; v < r.v1; v += kVecsChunk) {
          if (!SUM && !mbar_wait(&sh.full[written], write_phase, kWaitPolls, abort, status)) return false;
          for (int u = v + tid; p.d != nullptr && u < min(v + kVecsChunk, r.v1); u += kStep) {
            if (aligned) {
              __stcs(reinterpret_cast<uint4*>(d) + u, make_uint4(0, 0, 0, 0));
            } else {
              for (int w = 0; w < W; ++w) store_one<BF16>(d, int64_t(u) * W + w, 0.0f);
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.empty[written]);
          advance(written, write_phase);
        }
        return true;
      }
      const int own = int(r.label) - r.head;  // the label's place among the vectors' elements
      const Pair kk = pair_of(q.k, q.k), ss = pair_of(-q.shift, -q.shift), gg = pair_of(q.g, q.g);
#pragma unroll 1
      for (int v = r.v0; v < r.v1; v += kVecsChunk) {
        if (!SUM && !mbar_wait(&sh.full[written], write_phase, kWaitPolls, abort, status)) return false;
        const uint4* in = reinterpret_cast<const uint4*>(chunks + written * kStreamChunk) + tid;
        const int left = p.d == nullptr ? 0 : r.v1 - v - tid, mine = own - (v + tid) * W;
        uint4* to = reinterpret_cast<uint4*>(d) + v + tid;
#pragma unroll
        for (int j = 0; j < kThreadVecs; ++j) {
          if (j * kStep >= left) continue;
          float f[W];
          gradient_of<BF16>(in[j * kStep], kk, ss, gg, f);
          if (unsigned(mine - j * kStep * W) < unsigned(W)) {
#pragma unroll
            for (int w = 0; w < W; ++w)
              if (mine - j * kStep * W == w) f[w] += q.up;
          }
          if (aligned) {
            __stcs(to + j * kStep, narrow(f));
          } else {
#pragma unroll
            for (int w = 0; w < W; ++w) store_one<BF16>(reinterpret_cast<char*>(to + j * kStep), w, f[w]);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.empty[written]);
        advance(written, write_phase);
      }
      return true;
    };
    StreamRow before = {-1, -1, 0, 0, 0};
    for (int n = 0;; ++n) {
      if (!wait(sh.row_full, n, kStreamRows)) break;
      const StreamRow r = sh.row[n % kStreamRows];
      if (r.t >= 0 && SUM && !sum_row(n, r)) break;
      const bool late = SUM && WRITE;  // writes trail the sums by a row
      if (late && n > 0 && !write_row(n - 1, before)) break;
      if (!late && WRITE && r.t >= 0 && !write_row(n, r)) break;
      __syncwarp();
      if (lane == 0 && (late ? n > 0 : r.t >= 0)) mbar_arrive(&sh.row_free[(late ? n - 1 : n) % kStreamRows]);
      if (r.t < 0) break;
      before = r;
    }
  } else {
    // ---- finisher
    float mean = 0.0f;
    if (MODE == kPolicy) mean = mean_scale(p);
    int exchanges = 0;
    // The cluster's sum. The label's logit (x_label) goes with the owner's part of
    // it: where the gradient is written over the logits, the CTA that overwrites
    // that logit is the only one that reads it.
    auto join_cluster = [&](Lse z, int owner, float& x_label, bool& ok) {
      if (ranks == 1) return z;
      const int slot = exchanges % kStreamRows;
      if (lane == 0) mbar_arrive_expect_tx(&sh.cta_full[slot], 16 * ranks);
      if (lane < ranks)
        send_peer(&sh.cta_sum[slot][rank], &sh.cta_full[slot], lane, make_float4(z.c, z.s, x_label, 0.0f));
      ok = !__any_sync(~0u, !mbar_wait(&sh.cta_full[slot], (exchanges / kStreamRows) & 1, kWaitPolls, abort, status));
      ++exchanges;
      x_label = sh.cta_sum[slot][owner].z;
      Lse all = {sh.cta_sum[slot][0].x, sh.cta_sum[slot][0].y};
      for (int r = 1; r < ranks; ++r) all = lse_join(all, {sh.cta_sum[slot][r].x, sh.cta_sum[slot][r].y});
      return all;
    };
    const float nan = __int_as_float(0x7fffffff);
    // What a row needs from memory is read while the row before it is finished.
    struct Known {
      StreamRow r;
      int edge, owner;
      float edge_value, x_label, weight, adv, old, ref;
      float2 lse;
    };
    auto look_up = [&](int n, Known& q) {
      if (__any_sync(~0u, !wait(sh.row_full, n, kStreamRows))) return false;
      q.r = sh.row[n % kStreamRows];
      q.edge = -1;
      q.owner = 0;
      q.edge_value = -INFINITY;
      q.x_label = nan;
      q.weight = q.adv = q.old = q.ref = 0.0f;
      q.lse = make_float2(0.0f, 0.0f);
      const int64_t t = q.r.t;
      if (t < 0 || q.r.label < 0) return true;
      const char* x = row_of(t);
      const RowSpan<W, ES> span(x, int(p.vocab));
      if (rank == 0) q.edge = span.edge(lane);
      if (q.edge >= 0) q.edge_value = load_one<BF16>(x, q.edge);
      if (MODE == kPrefBackward) {
        q.lse = p.row_lse[t];
        q.weight = p.row_a[t];
        return true;
      }
      q.owner = span.owner(q.r.label, ranks);
      if (q.r.label < p.vocab && q.owner == rank) q.x_label = load_one<BF16>(x, q.r.label);
      if (MODE == kPolicy) {
        q.weight = p.row_a[t];
        q.adv = p.adv[t];
        q.old = p.old_logp[t];
      }
      if ((MODE == kPolicy || MODE == kPrefForward) && p.ref_logp != nullptr) q.ref = p.ref_logp[t];
      return true;
    };
    Known now, next;
    bool some = look_up(0, now);
    for (int n = 0; some && now.r.t >= 0; ++n, now = next) {
      some = look_up(n + 1, next);
      const StreamRow r = now.r;
      const int64_t t = r.t;
      StreamResult q = {p.k, 0.0f, 0.0f, 0.0f, 0};
      float terms[3] = {0.0f, 0.0f, 0.0f}, lp = 0.0f;
      const float edge_value = now.edge_value, weight = now.weight;
      const char* x = row_of(t);
      const int edge = now.edge;
      const bool teller = rank == 0 && lane == 0;
      bool ok = true;
      if (r.label >= 0) {
        if (MODE == kPrefBackward) {
          const float2 z = now.lse;  // the sign of 1 / sum tells the scale
          q.up = weight * p.inv_temp;
          q.k = z.y < 0.0f ? 1.0f : p.k;
          q.shift = z.x;
          q.g = -q.up * fabsf(z.y);
          q.zeros = weight == 0.0f;
        } else {
          ok = !__any_sync(~0u, !wait(sh.sum_full, n, kStreamRows));
          if (!ok) break;
          Lse z = {-INFINITY, 0.0f};
          if (lane < kStreamWarps) z = sh.warp_sum[n % kStreamRows][lane];
          auto with_edge = [&](Lse v, float k) {
            if (edge < 0) return v;
            const float c = fmaxf(-INFINITY, ceilf(edge_value * k));
            return lse_join(v, {c, exp2_approx(fmaf(edge_value, k, -finite_shift(c)))});
          };
          float x_label = now.x_label;
          z = join_cluster(lse_warp(with_edge(z, q.k), 32), now.owner, x_label, ok);
          if (!ok) break;
          // A sum below what kLeastShift may have cost it, once more from memory;
          // where x k itself is not finite (see rows_kernel), at k = 1.
          for (int again = 0; again < 2; ++again) {
            if (again == 0 ? !(z.s < 0.5f) : !isinf(z.c)) continue;
            if (again == 1) q.k = 1.0f;
            z = {-INFINITY, 0.0f};
            for (int v = r.v0 + lane; v < r.v1; v += 32)
              lse_add<BF16>(z, reinterpret_cast<const uint4*>(x + r.head * ES)[v], q.k);
            z = join_cluster(lse_warp(with_edge(z, q.k), 32), now.owner, x_label, ok);
            if (!ok) break;
          }
          if (!ok) break;
          const Two exact = log_prob(x_label, q.k, z);
          lp = exact.hi + exact.lo;
          q.shift = finite_shift(z.c);
          const float inv_sum = 1.0f / z.s;
          if (MODE == kPrefForward && teller) {
            // the log ratio before lp is rounded: sequences sum hundreds of them
            p.row_terms[t] = (exact.hi - now.ref) + exact.lo;
            p.row_lse[t] = make_float2(q.shift, copysignf(inv_sum, q.k == p.k ? 1.0f : -1.0f));
          }
          if (MODE == kPolicy) {
            const PolicyTerm term = policy_term(p, lp, weight, mean, now.adv, now.old, now.ref);
            for (int c = 0; c < 3; ++c) terms[c] = term.terms[c];
            q.zeros = weight == 0.0f;  // outside every sequence
            q.up = q.zeros ? 0.0f : r.label < p.vocab ? term.up : nan;
            q.g = -q.up * inv_sum;
          }
        }
      } else if (SUM) {
        ok = !__any_sync(~0u, !wait(sh.sum_full, n, kStreamRows));
        if (!ok) break;
      }
      if (SUM && teller) {
        p.logp[t] = lp;
        if (MODE == kPolicy)
          for (int c = 0; c < 3; ++c) p.row_terms[c * p.rows + t] = terms[c];
      }
      if (WRITE) {
        if (lane == 0) {
          sh.result[n % kStreamRows] = q;
          mbar_arrive(&sh.result_full[n % kStreamRows]);
        }
        if (p.d != nullptr) {
          char* d = static_cast<char*>(p.d) + t * p.dld * ES;
          if (r.label < 0) {
            const int zero = rank == 0 ? RowSpan<W, ES>(d, int(p.vocab)).edge(lane) : -1;
            if (zero >= 0) store_one<BF16>(d, zero, 0.0f);
          } else if (edge >= 0) {
            const float v = q.zeros ? 0.0f : exp2_approx(fmaf(edge_value, q.k, -q.shift)) * q.g;
            store_one<BF16>(d, edge, r.label == edge ? v + q.up : v);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.row_free[n % kStreamRows]);
    }
  }
  __syncwarp();
  if (ranks > 1) cluster_barrier();  // no CTA goes while another may still write to it
}

// The policy loss's statistics from the rows' terms.
__global__ void __launch_bounds__(1024) stats_kernel(LossParams p) {
  grid_dependency_wait();
  grid_dependents_launch();
  float out[3];
  sum_columns<1024, 3>(p.row_terms, p.rows, p.rows, out);
  if (threadIdx.x == 0) {
    p.stats[0] = p.kl > 0.0f ? out[0] + p.kl * out[1] : out[0];
    p.stats[1] = out[0];
    p.stats[2] = out[1];
    p.stats[3] = out[2];
  }
}

// ---------------------------------------------------------------- pairs

// One CTA a pair: the log ratios of its two sequences, the loss of the pair
// and the coefficient of each of its rows; the last one sums the statistics.
__global__ void __launch_bounds__(256) pair_kernel(LossParams p) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t pairs = p.n_seq / 2, i = blockIdx.x;
  __shared__ Two sums[2][8];
  __shared__ int counts[2][8];
  __shared__ bool last;
  int64_t bounds[3];
  for (int h = 0; h < 3; ++h) bounds[h] = seq_bound(p, 2 * i + h);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  // Sums of log ratios in pairs of fp32 (fp64 adds are slow here).
  for (int h = 0; h < 2; ++h) {
    Two a = {0.0f, 0.0f};
    int n = 0;
#pragma unroll 4
    for (int64_t t = bounds[h] + threadIdx.x; t < bounds[h + 1]; t += 256)
      if (p.labels[t] >= 0) {
        a = add_two(a, p.row_terms[t], 0.0f);
        ++n;
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a = add_two(a, __shfl_xor_sync(~0u, a.hi, o), __shfl_xor_sync(~0u, a.lo, o));
    n = __reduce_add_sync(~0u, n);
    if (lane == 0) sums[h][warp] = a, counts[h][warp] = n;
  }
  __syncthreads();
  __shared__ float coef[2];
  if (threadIdx.x == 0) {
    Two sum[2];
    int n[2];
    for (int h = 0; h < 2; ++h) {
      sum[h] = sums[h][0];
      n[h] = counts[h][0];
      for (int w = 1; w < 8; ++w) sum[h] = add_two(sum[h], sums[h][w].hi, sums[h][w].lo), n[h] += counts[h][w];
    }
    const PairTerms r = pair_terms(p, sum, n);
    float* terms = p.row_terms + p.rows;
    for (int h = 0; h < 2; ++h) {
      p.ratios[2 * i + h] = r.ratio[h];
      coef[h] = r.coef[h];
    }
    for (int c = 0; c < 4; ++c) terms[c * pairs + i] = r.terms[c];
    __threadfence();
    last = atomicAdd(&p.tickets[0], 1u) == gridDim.x - 1;
  }
  __syncthreads();
  for (int h = 0; h < 2; ++h)
    for (int64_t t = bounds[h] + threadIdx.x; t < bounds[h + 1]; t += 256) p.row_a[t] = coef[h];
  if (i == 0)
    for (int64_t t = threadIdx.x; t < bounds[0]; t += 256) p.row_a[t] = 0.0f;
  if (i == pairs - 1)
    for (int64_t t = bounds[2] + threadIdx.x; t < p.rows; t += 256) p.row_a[t] = 0.0f;
  if (!last) return;
  __threadfence();
  float out[4];
  sum_columns<256, 4>(p.row_terms + p.rows, pairs, pairs, out);
  if (threadIdx.x == 0)
    for (int c = 0; c < 4; ++c) p.stats[c] = out[c];
}

// ---------------------------------------------------------------- launches

// Launched so that it may be scheduled while the kernel before it drains; every
// kernel here waits for that one before it touches memory.
cudaError_t launch_after(void (*kernel)(LossParams), const LossParams& p, int64_t grid, int threads, int cluster,
                         cudaStream_t stream, size_t smem = 0) {
  if (grid <= 0) return cudaSuccess;
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(grid));
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// How many clusters of the streaming kernel run at once on the current device.
cudaError_t active_clusters(const void* kernel, int cluster, size_t smem, int* workers) {
  static std::mutex mu;
  static std::vector<std::array<int, 3>> known;  // device, cluster, workers (the same for every kernel of its shape)
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  std::lock_guard<std::mutex> lock(mu);
  for (const auto& k : known)
    if (k[0] == dev && k[1] == cluster) {
      *workers = k[2];
      return cudaSuccess;
    }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(device_sms() / cluster * cluster));
  cfg.blockDim = dim3(kStreamThreads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(cluster);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  err = cudaOccupancyMaxActiveClusters(workers, kernel, &cfg);
  if (err != cudaSuccess) return err;
  if (*workers < 1) return cudaErrorInvalidConfiguration;
  known.push_back({dev, cluster, *workers});
  return cudaSuccess;
}

// Calls with many long rows stream them; the others take a cluster a row.
// Measured, a cluster a row against streaming (log-probabilities / policy loss,
// in a graph of calls): 6000 rows of 24 KB 41 / 73 and 60 / 96 us, of 32 KB
// 43 / 81 and 61 / 98, of 40 KB (where a row needs 512 threads) 90 / 138 and
// 62 / 111, of 56 KB 93 / 151 and 63 / 121; rows of 64 KB, 300 of them 5.9 / 12.5
// and 5.5 / 11.7, 600 of them 10.2 / 20.9 and 8.5 / 17.9, 1200 of them 19.4 / 40.5
// and 14.5 / 33.4.
constexpr int64_t kStreamRowBytes = 32768, kStreamRowsAnSm = 4;

template <bool BF16, int MODE>
cudaError_t launch_rows_typed(LossParams p, cudaStream_t stream) {
  const int64_t bytes = p.vocab * (BF16 ? 2 : 4), vecs = (bytes + 15) / 16, sms = device_sms();
  p.cluster = 1;
  while (MODE == kPolicy && p.cluster < kMaxCluster && bytes > int64_t(kStreamSlice) * p.cluster) p.cluster *= 2;
  if (bytes > kStreamRowBytes && (MODE != kPolicy || bytes <= int64_t(kStreamSlice) * p.cluster) && p.rows * p.cluster >= kStreamRowsAnSm * sms && !p.few) {
    void (*kernel)(LossParams) = stream_kernel<BF16, MODE>;
    constexpr size_t kSmem = size_t(kStreamChunks) * kStreamChunk + 128;
    cudaError_t err = status_ref(&p.status_word, &p.status_host);
    if (err == cudaSuccess)
      err = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel), cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmem));
    int workers = int(sms);
    if (err == cudaSuccess && p.cluster > 1) err = active_clusters(reinterpret_cast<const void*>(kernel), p.cluster, kSmem, &workers);
    if (err != cudaSuccess) return err;
    return launch_after(kernel, p, std::min<int64_t>(workers, p.rows) * p.cluster, kStreamThreads, p.cluster, stream, kSmem);
  }
  // The smallest CTA, then the smallest cluster, that holds a row; a few rows
  // are spread over more CTAs, so that every SM has some.
  const int threads = vecs <= 128 * kVecs ? 128 : vecs <= 256 * kVecs ? 256 : 512;
  p.cluster = 1;
  while (p.cluster < kMaxCluster && vecs > int64_t(threads) * kVecs * p.cluster) p.cluster *= 2;
  while (p.cluster < kMaxCluster && p.rows * p.cluster * 2 <= 2 * sms && vecs >= int64_t(threads) * 2 * p.cluster)
    p.cluster *= 2;
  while (p.cluster > 1 && p.rows * p.cluster > 0x7fffffff) p.cluster /= 2;
  void (*kernel)(LossParams) = threads == 128   ? rows_kernel<BF16, MODE, 128>
                               : threads == 256 ? rows_kernel<BF16, MODE, 256>
                                                : rows_kernel<BF16, MODE, 512>;
  return launch_after(kernel, p, p.rows * p.cluster, threads, p.cluster, stream);
}

template <int MODE>
cudaError_t launch_rows(const LossParams& p, ar_dtype dtype, cudaStream_t stream) {
  return dtype == AR_BF16 ? launch_rows_typed<true, MODE>(p, stream) : launch_rows_typed<false, MODE>(p, stream);
}

}  // namespace

cudaError_t launch_token_logp(const LossParams& p, ar_dtype dtype, cudaStream_t stream) {
  return launch_rows<kLogp>(p, dtype, stream);
}

cudaError_t launch_policy_loss(const LossParams& q, ar_dtype dtype, cudaStream_t stream) {
  LossParams p = q;
  p.few = p.rows <= kFewRows && p.n_seq <= kFewSequences;
  if (p.rows == 0) return cudaMemsetAsync(p.stats, 0, 16, stream);
  cudaError_t err = p.few ? cudaSuccess : launch_after(count_kernel, p, p.n_seq, 256, 1, stream);
  if (err == cudaSuccess) err = launch_rows<kPolicy>(p, dtype, stream);
  if (err == cudaSuccess) err = launch_after(stats_kernel, p, 1, 1024, 1, stream);
  return err;
}

cudaError_t launch_preference_loss(const LossParams& q, ar_dtype dtype, cudaStream_t stream) {
  LossParams p = q;
  p.few = p.rows > 0 && p.rows <= kFewRows && p.n_seq <= kFewSequences && p.d != nullptr;
  cudaError_t err = p.rows == 0 ? cudaMemsetAsync(p.tickets, 0, 4, stream) : launch_rows<kPrefForward>(p, dtype, stream);
  if (err == cudaSuccess && !p.few) err = launch_after(pair_kernel, p, p.n_seq / 2, 256, 1, stream);
  if (err == cudaSuccess && p.d != nullptr) err = launch_rows<kPrefBackward>(p, dtype, stream);
  return err;
}

}  // namespace ar
