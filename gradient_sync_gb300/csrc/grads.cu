// The global norm of many gradient tensors, clipping, and the AdamW step.
//
// norm:   N = sqrt(sum over all tensors of |s g|^2), or the largest |s g|;
//         c = min(1, max_norm / (N + eps))
// clip:   out = (c s) g
// AdamW:  M' = b1 M + (1 - b1) G, V' = b2 V + (1 - b2) G^2, G = (c s) g,
//         W' = (1 - lr wd) W - lr / (1 - b1^t) M' / (sqrt(V' / (1 - b2^t)) + eps)
//
// All of it is bound by HBM where there is much, by launches where there is
// little: two to six operations an element against 2 to 32 bytes.
//
// A list of tensors is one sequence of granules, 16 aligned bytes each, and a
// warp takes a stretch of it: whatever the tensors' sizes, every warp has equal
// work, and a tensor's sum is that of the stretches it lies in. A stretch and a
// tensor meet at most once, so that the sum of warp w over tensor i has a place
// of its own, w + i, and nothing is added in an order that timing could change.
//
// Sums of squares are pairs of fp32 numbers, about 46 bits (one fp64 operation takes
// a warp some 200 cycles here: joins in fp64 cost more than the reading), in
// three bands of magnitude, each at its own power of two, so that finite elements of
// any size have their norm.
#include "grads.h"

#include <algorithm>

#include "common.cuh"
#include "pairs.cuh"

namespace ar {
namespace {

constexpr int kNormThreads = 512;
constexpr int kLoads = 8;  // 16-byte loads in flight a thread

__device__ __forceinline__ uint4 load16(const char* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

// The same with a priority for staying in the L2. Of a list that is to be clipped, the norm keeps the last granules of
// every stretch, kKept bytes in all, and the scaling, which goes through a stretch from its end, lets them go: 67 M fp32
// elements 131 -> 125 us, in place 123 -> 118, 9 M 20.2 -> 18.6. (28, 55, 80 and 110 MB kept, before the scaling let go of lines: 128, 124.5,
// 123.5 and 124.7 us.) Lines have the priority until it is taken from them, whatever reads them later: with it, six passes
// over other 80 MB took 129 us behind any such call, 105 without. It is taken where nothing is scaled too, which is 4 us
// of a call in place that does not clip.
constexpr int64_t kKept = int64_t(80) << 20;
__device__ __forceinline__ uint64_t keep_policy() {
  uint64_t p;
  asm("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ uint64_t leave_policy() {
  uint64_t p;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ uint4 load16(const char* p, uint64_t policy) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.L2::cache_hint.v4.u32 {%0, %1, %2, %3}, [%4], %5;"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p), "l"(policy));
  return r;
}

// A sum of squares v * 2^(176 band), or, of maxima, a magnitude (band 0). An
// infinity among the elements is the band kInf, a NaN kNan: the higher band is
// what a join keeps (the lower one's share is below 2^-46 of it, but
// for the bottom of a band, where it is added).
enum Band : int { kSmall = -1, kMid = 0, kBig = 1, kInf = 2, kNan = 3 };
struct Value {
  int band;
  Two v;
};
constexpr float kScale = 3.0948500982134507e26f;      // 2^88
constexpr float kUnscale = 3.2311742677852644e-27f;   // 2^-88
constexpr float kMidLow = 8.0779356694631609e-28f;    // 2^-90: where a batch's fp32 squares have lost nothing
constexpr float kMidHigh = 1.2379400392853803e27f;    // 2^90: where 2^34 batches still fit
__device__ __forceinline__ Two lowered(Two v) { return {v.hi * kUnscale * kUnscale, v.lo * kUnscale * kUnscale}; }
__device__ __forceinline__ Value sum_of(Value a, Value b) {
  if (a.band == b.band) return {a.band, add(a.v, b.v)};
  const Value& top = a.band > b.band ? a : b;
  const Value& low = a.band > b.band ? b : a;
  return {top.band, top.band - low.band == 1 && top.band <= kBig ? add(top.v, lowered(low.v)) : top.v};
}
__device__ __forceinline__ Value larger(Value a, Value b) { return a.band > b.band || (a.band == b.band && a.v.hi >= b.v.hi) ? a : b; }
template <bool MAX>
__device__ __forceinline__ Value join(Value a, Value b) {
  return MAX ? larger(a, b) : sum_of(a, b);
}
__device__ __forceinline__ Value nothing() { return {kSmall, {0.0f, 0.0f}}; }

// A magnitude by its bits.
__device__ __forceinline__ Value magnitude(uint32_t bits) {
  if (bits >= 0x7f800000u) return {bits > 0x7f800000u ? kNan : kInf, {0.0f, 0.0f}};
  return {kMid, {__uint_as_float(bits), 0.0f}};
}

template <bool MAX>
__device__ __forceinline__ Value warp_join(Value a) {
  if (MAX) {
    const uint32_t top = __reduce_max_sync(~0u, a.band == kMid ? __float_as_uint(a.v.hi) : a.band < kMid ? 0u : a.band == kInf ? 0x7f800000u : 0x7fc00000u);
    return magnitude(top);
  }
  // (the bands mostly agree, but for lanes that have nothing)
  const int top = __reduce_max_sync(~0u, a.band);
  if (a.v.hi == 0.0f && a.band < kInf) a.band = top;
  if (__reduce_min_sync(~0u, a.band) == top) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a.v = add(a.v, {__shfl_xor_sync(~0u, a.v.hi, o), __shfl_xor_sync(~0u, a.v.lo, o)});
    return a;
  }
#pragma unroll 1
  for (int o = 16; o > 0; o >>= 1)
    a = sum_of(a, {__shfl_xor_sync(~0u, a.band, o), {__shfl_xor_sync(~0u, a.v.hi, o), __shfl_xor_sync(~0u, a.v.lo, o)}});
  return a;
}

// One square, in its band.
__device__ __forceinline__ Value square(float x) {
  const float a = fabsf(x);
  if (!(a < INFINITY)) return {a == INFINITY ? kInf : kNan, {0.0f, 0.0f}};
  const float f = a < 1e-13f ? kScale : a > 1e13f ? kUnscale : 1.0f, b = a * f;
  return {a < 1e-13f ? kSmall : a > 1e13f ? kBig : kMid, {b * b, fmaf(b, b, -(b * b))}};
}

// The sum of squares of a batch whose fp32 squares could have overflowed, or have
// been lost below fp32's range, from memory again.
template <bool BF16>
__device__ __noinline__ Value squares_in_bands(const char* base, int64_t g, int64_t hi) {
  Value s = nothing();
#pragma unroll 1
  for (int i = 0; i < kLoads && g < hi; ++i, g += 32) {
    const uint4 r = load16(base + 16 * g);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll 1
    for (int j = 0; j < 4; ++j) {
      s = sum_of(s, square(BF16 ? bf16lo(w[j]) : __uint_as_float(w[j])));
      if (BF16) s = sum_of(s, square(bf16hi(w[j])));
    }
  }
  return s;
}

// Adds the sum of squares of a batch, the granules g, g + 32, ... below hi, to a
// sum: fp32 within it (at most 64 terms). `odd`: of batches outside the middle band.
template <bool BF16>
__device__ __forceinline__ void add_squares(const uint4 (&r)[kLoads], const char* base, int64_t g, int64_t hi, Two& mid, Value& odd) {
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  uint32_t any = 0;
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const uint32_t w[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float a = BF16 ? bf16lo(w[j]) : __uint_as_float(w[j]);
      s[j] = fmaf(a, a, s[j]);
      if (BF16) s[j] = fmaf(bf16hi(w[j]), bf16hi(w[j]), s[j]);
      any |= w[j];
    }
  }
  const float sum = (s[0] + s[1]) + (s[2] + s[3]);
  if (sum >= kMidLow && sum < kMidHigh) mid = add(mid, {sum, 0.0f});
  else if ((any & (BF16 ? 0x7fff7fffu : 0x7fffffffu)) != 0) odd = sum_of(odd, squares_in_bands<BF16>(base, g, hi));
}

// Magnitudes as integers order like the numbers, NaN above infinity.
template <bool BF16>
__device__ __forceinline__ uint32_t largest(const uint4 (&r)[kLoads], uint32_t top) {
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const uint32_t w[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (BF16) {
        top = max(top, (w[j] << 16) & 0x7fffffffu);
        top = max(top, w[j] & 0x7fff0000u);
      } else {
        top = max(top, w[j] & 0x7fffffffu);
      }
    }
  }
  return top;
}

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
// The same place in another CTA of the cluster.
template <class T>
__device__ __forceinline__ T* peer(T* p, int rank) {
  uint64_t a;
  asm("mapa.u64 %0, %1, %2;" : "=l"(a) : "l"(p), "r"(rank));
  return reinterpret_cast<T*>(a);
}

// A tensor as granules: `lead` elements of the first one lie before it.
struct Span {
  const char* base;  // of granule 0
  int64_t count, granules, full;  // granules below `full` end inside the tensor
  int es, lead;
  __device__ Span(const char* p, int64_t count_kind) {
    count = count_kind >> 1;
    es = (count_kind & 1) ? 2 : 4;
    const int off = int(reinterpret_cast<uintptr_t>(p) & 15);
    base = p - off;
    lead = off / es;
    granules = ((lead + count) * es + 15) >> 4;
    full = ((lead + count) * es) >> 4;
  }
  // The elements that are not in whole granules, one a lane (-1: none).
  __device__ int64_t edge(int64_t g0, int64_t g1, int lane) const {
    const int per = 16 / es;
    const int64_t head = lead > 0 ? min(count, int64_t(per - lead)) : 0;
    const int64_t tail = max(head, full * per - lead);
    if (lane < per) return g0 == 0 && lane < head ? lane : -1;
    const int64_t e = tail + lane - per;
    return g1 == granules && e < count && lane < 2 * per ? e : -1;
  }
};

__device__ __forceinline__ float element(const char* p, int64_t e, int es) {
  return es == 2 ? bf16_to_f32(reinterpret_cast<const uint16_t*>(p)[e]) : reinterpret_cast<const float*>(p)[e];
}

// The entry that a granule (or tile) lies in, by a warp: of 32 entries at a time, through ordinary loads (from the
// constant bank, every step of a bisection is a miss of its own).
template <class Table>
__device__ __forceinline__ int entry_of(const Table& t, int64_t g, int lane) {
  const Table* p = &t;
  asm("" : "+l"(p));
  int lo = 0, hi = t.n;  // the entry is in [lo, hi)
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, at = lo + lane * step;
    const unsigned not_behind = __ballot_sync(~0u, at < hi && p->e[at].first <= g);
    lo += (31 - __clz(int(not_behind))) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// What a tensor costs a warp beside its granules, in granules: a list counts as that much longer, so that no
// warp has many short tensors to go through, one after the other. (Clipping of 309 uneven tensors, 35 MB: 35.0 us
// with 0, 26.7 with 64, 21.5 with 192, 18.8 with 512, 19.1 with 1024.)
constexpr int kTensorGranules = 512;
// Granules a warp: a multiple of 32, so that its loads are whole lines.
inline int64_t stretch(int64_t granules, int64_t warps) { return (granules + warps * 32 - 1) / (warps * 32) * 32; }
// The warp that a granule belongs to. (2^37 granules, 2 TB, are more than any device has.)
__device__ __forceinline__ int warp_of(int64_t granule, int64_t per) { return int(uint32_t(granule >> 5) / uint32_t(per >> 5)); }

// KEEP: granules from `kept` on stay in the L2.
template <bool BF16, bool MAX, bool KEEP>
__device__ __forceinline__ Value value_of(const char* base, int64_t lo, int64_t hi, int lane, int64_t kept) {
  Two mid = {0.0f, 0.0f};
  Value odd = nothing();
  uint32_t top = 0;
  uint4 r[kLoads];
  int64_t g = lo + lane;
  const uint64_t keep = KEEP ? keep_policy() : 0, leave = KEEP ? leave_policy() : 0;
  const auto take = [&] {
    if (MAX) top = largest<BF16>(r, top);
    else add_squares<BF16>(r, base, g, hi, mid, odd);
  };
#pragma unroll 1
  for (; g + 32 * (kLoads - 1) < hi; g += 32 * kLoads) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      r[i] = KEEP ? load16(base + 16 * (g + 32 * i), g >= kept ? keep : leave) : load16(base + 16 * (g + 32 * i));
    take();
  }
  if (g < hi) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) r[i] = g + 32 * i < hi ? load16(base + 16 * (g + 32 * i)) : make_uint4(0, 0, 0, 0);
    take();
  }
  if (MAX) return magnitude(top);
  return mid.hi > 0.0f ? sum_of(odd, {kMid, mid}) : odd;
}

// Every warp's sum over each tensor that its stretch [lo, hi) meets: place(i) for tensor i.
template <bool MAX, bool KEEP, class Table, class Place>
__device__ __forceinline__ void stretch_values(const Table& t, int64_t lo, int64_t hi, int lane, Place place) {
  if (lo >= hi) return;
#pragma unroll 1
  for (int i = entry_of(t, lo, lane); i < t.n && t.e[i].first < hi; ++i) {
    const Span s(t.e[i].in, t.e[i].count);
    const int64_t g0 = max(lo - t.e[i].first, int64_t(0)), g1 = min(hi - t.e[i].first, s.granules);
    if (g0 >= g1) continue;
    const int64_t a = max(g0, int64_t(s.lead > 0)), b = min(g1, s.full);
    const int64_t kept = hi - t.keep - t.e[i].first;
    Value v = s.es == 2 ? value_of<true, MAX, KEEP>(s.base, a, b, lane, kept) : value_of<false, MAX, KEEP>(s.base, a, b, lane, kept);
    const int64_t e = s.edge(g0, g1, lane);
    if (e >= 0) {
      const float x = element(t.e[i].in, e, s.es);
      v = MAX ? larger(v, magnitude(__float_as_uint(x) & 0x7fffffffu)) : x != 0.0f ? sum_of(v, square(x)) : v;
    }
    v = warp_join<MAX>(v);
    if (lane == 0) *place(i) = v;
  }
}

// The warps' sums over the tensors that a CTA's stretch meets, joined: one sum a CTA and tensor, at job.partials[CTA + tensor].
// Bound by HBM: 1.14 G bf16 elements in 206 tensors 317 us, 7.2 TB/s; 67 M fp32 45 us, 6.0 TB/s (start and end of a
// launch). Two CTAs an SM with 8 loads of 16 bytes a thread are 128 KB in flight; 2048 CTAs in place of 304 gained
// nothing (332 us, and the end has more sums to join).
template <int CAP, bool MAX, bool KEEP>
__global__ void __launch_bounds__(kNormThreads) norm_kernel(const __grid_constant__ GradTable<CAP> t, GradJob job) {
  constexpr int kWarps = kNormThreads / 32;
  grid_dependency_wait();
  grid_dependents_launch();
  __shared__ Value part[kWarps + CAP];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t from = int64_t(blockIdx.x) * kWarps * t.per, to = min(t.granules, from + kWarps * t.per);
  const int64_t lo = from + warp * t.per, hi = min(t.granules, lo + t.per);
  if (from >= to) return;
  const int first = entry_of(t, from, lane);
  stretch_values<MAX, KEEP>(t, lo, hi, lane, [&](int i) { return part + (warp + i - first); });
  __syncthreads();
  Value* partials = reinterpret_cast<Value*>(job.partials) + blockIdx.x;
#pragma unroll 1
  for (int i = first + warp; i < t.n && t.e[i].first < to; i += kWarps) {
    const Span s(t.e[i].in, t.e[i].count);
    const int64_t g0 = max(from, t.e[i].first), g1 = min(to, t.e[i].first + s.granules);
    if (g0 >= g1) continue;
    const int w = warp_of(g0 - from, t.per) + lane;
    const Value v = warp_join<MAX>(w <= warp_of(g1 - 1 - from, t.per) ? part[w + i - first] : nothing());
    if (lane == 0) partials[i] = v;
  }
}

// The root of a sum of squares as two numbers (times 2^(88 band)).
__device__ __forceinline__ Two root_of(Two v) {
  if (!(v.hi > 0.0f)) return {0.0f, 0.0f};
  const float r = sqrtf(v.hi);
  return {r, (fmaf(-r, r, v.hi) + v.lo) / (2.0f * r)};
}
__device__ __forceinline__ float power(int band) { return band == kBig ? kScale : band == kSmall ? kUnscale : 1.0f; }

// A sum's norm, in fp32.
template <bool MAX>
__device__ __forceinline__ float norm_of(Value v, float scale) {
  if (v.band >= kInf) return v.band == kInf ? INFINITY : __int_as_float(0x7fc00000);
  const Two r = MAX ? v.v : root_of(v.v);
  // (one of the two factors may leave fp32's range where the norm does not)
  const float f = MAX ? 1.0f : power(v.band);
  return fabsf(scale) >= 1.0f == f >= 1.0f ? (r.hi + r.lo) * f * scale : (r.hi + r.lo) * (f * scale);
}

template <bool MAX>
__device__ __forceinline__ void write_stats(const GradJob& job, Value total) {
  const bool finite = total.band < kInf;
  const float scale = fabsf(job.grad_scale);
  float c = 0.0f;
  if (finite) {
    // max_norm / (r scale + eps), all in pairs and times f
    Two r = MAX ? total.v : root_of(total.v);
    float f = MAX ? 1.0f : 1.0f / power(total.band);
    if (MAX && r.hi > 1e18f) f = kUnscale, r = {r.hi * f, 0.0f};
    const float p = r.hi * scale;
    r = two_sum(p, fmaf(r.hi, scale, -p) + r.lo * scale);
    const Two n = add(r, {job.eps * f, job.eps_low * f}), m = {job.max_norm * f, job.max_norm_low * f};
    c = m.hi / n.hi;
    if (c < INFINITY) c += ((fmaf(-c, n.hi, m.hi) + m.lo) - c * n.lo) / n.hi;
    if (!(c < 1.0f)) c = p < INFINITY ? 1.0f : 0.0f;  // (1 also for 0 / 0: a norm of 0 and no eps)
  }
  job.stats[0] = norm_of<MAX>(total, scale);
  job.stats[1] = c;
  job.stats[2] = c < 1.0f ? 1.0f : 0.0f;
  job.stats[3] = finite ? 1.0f : 0.0f;
}

// The tensors' norms from the sums in `part`, each of `per` granules, by one CTA; returns the sum over all tensors
// (thread 0). A lane a tensor, but for tensors of many sums.
template <bool MAX, class Table>
__device__ __forceinline__ Value finish_tensors(const Table& table, int64_t per, const GradJob& job, const Value* part, Value* sums) {
  constexpr int kFew = 4;
  const Table* t = &table;
  asm("" : "+l"(t));  // (ordinary loads: lanes read entries of their own)
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = int(blockDim.x) / 32;
  const float scale = fabsf(job.grad_scale);
  Value mine = nothing();
#pragma unroll 1
  for (int i0 = 0; i0 < t->n; i0 += 32 * warps) {
    const int i = i0 + lane * warps + warp;  // (tensors beside one another are often alike: to different warps)
    int from = 0, to = 0;  // of the tensor's sums
    if (i < t->n && t->e[i].count > 1) {
      const int64_t first = t->e[i].first;
      from = warp_of(first, per) + i;
      to = warp_of(first + Span(t->e[i].in, t->e[i].count).granules - 1, per) + i + 1;
    }
    Value v = nothing();
    if (to - from <= kFew)
      for (int j = from; j < to; ++j) v = join<MAX>(v, part[j]);
    unsigned many = __ballot_sync(~0u, to - from > kFew);
    while (many != 0) {
      const int owner = __ffs(int(many)) - 1;
      many &= many - 1;
      const int last = __shfl_sync(~0u, to, owner);
      Value w = nothing();
      for (int j = __shfl_sync(~0u, from, owner) + lane; j < last; j += 32) w = join<MAX>(w, part[j]);
      w = warp_join<MAX>(w);
      if (lane == owner) v = w;
    }
    if (i < t->n && job.norms != nullptr) job.norms[i] = norm_of<MAX>(v, scale);
    mine = join<MAX>(mine, v);
  }
  mine = warp_join<MAX>(mine);
  if (lane == 0) sums[warp] = mine;
  __syncthreads();
  if (warp == 0) mine = warp_join<MAX>(lane < warps ? sums[lane] : nothing());
  return mine;
}

// One CTA; behind the last launch of a call, the statistics. Bound by latency: 6 us with cold caches for 300 tensors (51 in
// fp64, a warp a tensor).
template <int CAP, bool MAX>
__global__ void __launch_bounds__(1024) finish_kernel(const __grid_constant__ GradTable<CAP> t, GradJob job, int group, int groups) {
  grid_dependency_wait();
  grid_dependents_launch();
  extern __shared__ __align__(16) char shared[];
  Value* part = reinterpret_cast<Value*>(shared);
  __shared__ Value sums[32];
  const int64_t per = t.per * (kNormThreads / 32);
  const int used = t.granules > 0 ? warp_of(t.granules - 1, per) + t.n : 0;
  for (int i = threadIdx.x; i < used; i += 1024) part[i] = reinterpret_cast<const Value*>(job.partials)[i];
  __syncthreads();
  Value total = finish_tensors<MAX>(t, per, job, part, sums);
  if (threadIdx.x == 0) {
    Value* all = reinterpret_cast<Value*>(job.groups);
    if (group + 1 < groups) {
      all[group] = total;
    } else {
      for (int i = 0; i < group; ++i) total = join<MAX>(total, all[i]);
      write_stats<MAX>(job, total);
    }
  }
}

template <bool BF16>
__device__ __forceinline__ uint4 scaled(const uint4& r, float f) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    o[j] = BF16 ? pack_bf16x2(bf16lo(w[j]) * f, bf16hi(w[j]) * f) : __float_as_uint(__uint_as_float(w[j]) * f);
  return make_uint4(o[0], o[1], o[2], o[3]);
}

__device__ __forceinline__ void store_element(char* p, int64_t e, int es, float v) {
  if (es == 2) reinterpret_cast<uint16_t*>(p)[e] = f32_to_bf16(v);
  else reinterpret_cast<float*>(p)[e] = v;
}

// Takes from granules [lo, hi) the priority for staying in the L2.
__device__ __forceinline__ void let_go(const char* base, int64_t lo, int64_t hi, int lane) {
  for (int64_t g = lo + 8 * lane; g < hi + 7; g += 8 * 32) {  // (a line is 8 granules, and begins anywhere)
    const uint64_t line = reinterpret_cast<uint64_t>(base + 16 * min(g, hi - 1)) & ~uint64_t(127);
    asm volatile("applypriority.global.L2::evict_normal [%0], 128;" ::"l"(line) : "memory");
  }
}

// Granules [lo, hi) of a tensor, times f; `zero`: zeros, whatever they hold.
template <bool BF16>
__device__ __forceinline__ void scale_granules(const char* base, char* out, int64_t lo, int64_t hi, int lane, float f,
                                               bool zero) {
  // From the end: what the norm has kept in the L2.
  const uint64_t leave = leave_policy();
  for (int64_t n = (hi - lo + 32 * kLoads - 1) / (32 * kLoads); n > 0; --n) {
    const int64_t g = lo + (n - 1) * 32 * kLoads + lane;
    uint4 r[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      r[i] = g + 32 * i < hi && !zero ? load16(base + 16 * (g + 32 * i), leave) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      if (g + 32 * i < hi) __stcs(reinterpret_cast<uint4*>(out + 16 * (g + 32 * i)), scaled<BF16>(r[i], f));
  }
}

// The stretch [lo, hi), scaled, from its end.
template <class Table>
__device__ __forceinline__ void scale_stretch(const Table& t, int64_t lo, int64_t hi, int lane, float f, bool zero) {
  if (lo >= hi) return;
#pragma unroll 1
  for (int i = entry_of(t, hi - 1, lane); i >= 0; --i) {
    const GradEntry& e = t.e[i];
    const Span s(e.in, e.count);
    const int64_t g0 = max(lo - e.first, int64_t(0)), g1 = min(hi - e.first, s.granules);
    if (g0 < g1 && !(f == 1.0f && e.in == e.out)) {
      if (((e.in - e.out) & 15) == 0) {
        const int64_t a = max(g0, int64_t(s.lead > 0)), b = min(g1, s.full);
        char* out = e.out - s.lead * s.es;
        if (s.es == 2) scale_granules<true>(s.base, out, a, b, lane, f, zero);
        else scale_granules<false>(s.base, out, a, b, lane, f, zero);
        const int64_t x = s.edge(g0, g1, lane);
        if (x >= 0) store_element(e.out, x, s.es, zero ? 0.0f : element(e.in, x, s.es) * f);
      } else {
        const int p = 16 / s.es;
        const int64_t from = max(g0 * p - s.lead, int64_t(0)), to = min(g1 * p - s.lead, s.count);
#pragma unroll 8
        for (int64_t x = from + lane; x < to; x += 32)
          store_element(e.out, x, s.es, zero ? 0.0f : element(e.in, x, s.es) * f);
      }
    }
    if (t.keep > 0) {  // (whatever has been read)
      const int64_t kept = max(g0, hi - t.keep - e.first);
      if (kept < g1) let_go(s.base, kept, g1, lane);
    }
    if (e.first <= lo) break;
  }
}

// The scaled gradients, stretch by stretch as the norm read them. Bound by HBM: 67 M fp32 elements 84 us with cold
// caches, 6.4 TB/s; the clipping of them 125 us in all. (A batch of loads a warp, CTAs from the end of the list on:
// 136 us in place of 129, before the L2 was told what to keep.)
template <int CAP>
__global__ void __launch_bounds__(kNormThreads, 2) scale_kernel(const __grid_constant__ GradTable<CAP> t, GradJob job) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t w = int64_t(blockIdx.x) * (kNormThreads / 32) + threadIdx.x / 32;
  const bool zero = job.stats[3] == 0.0f;
  scale_stretch(t, w * t.per, min(t.granules, (w + 1) * t.per), threadIdx.x % 32, zero ? 0.0f : job.stats[1] * job.grad_scale, zero);
}

// A short list, by one cluster in one launch: the warps' sums, the statistics, and, CLIP, the scaled gradients. Bound by
// latency: an adapter's 139 KB 5.3 us in a graph of calls, clipping 8.5; clusters of up to 8 CTAs with at most 4 loads a lane,
// against 16 loads, 5.4 and 5.9 us, clipping 7.6 and 9.6.
constexpr int kMaxRanks = 8;
template <bool MAX, bool CLIP>
__global__ void __launch_bounds__(kNormThreads) short_kernel(const __grid_constant__ GradTable<kGradCapSmall> t, GradJob job) {
  grid_dependency_wait();
  grid_dependents_launch();
  __shared__ Value part[kMaxRanks * (kNormThreads / 32) + kGradCapSmall], sums[32];
  __shared__ float factor;
  const int lane = threadIdx.x % 32, ranks = int(gridDim.x), rank = int(blockIdx.x);
  const int w = rank * (kNormThreads / 32) + threadIdx.x / 32;
  const int64_t lo = w * t.per, hi = min(t.granules, lo + t.per);
  if (ranks > 1) cluster_barrier();  // (the first CTA runs)
  // the first CTA's shared memory has all sums
  Value* to = ranks > 1 ? peer(part, 0) : part;
  stretch_values<MAX, false>(t, lo, hi, lane, [&](int i) { return to + (w + i); });
  if (ranks > 1) cluster_barrier();
  else __syncthreads();
  if (rank == 0) {
    const Value total = finish_tensors<MAX>(t, t.per, job, part, sums);
    if (threadIdx.x == 0) {
      write_stats<MAX>(job, total);
      factor = total.band >= kInf ? 0.0f : job.stats[1] * job.grad_scale;
      sums[0].band = total.band;
    }
  }
  if (!CLIP) return;
  if (ranks > 1) cluster_barrier();
  else __syncthreads();
  const float f = ranks > 1 ? *peer(&factor, 0) : factor;
  const bool zero = (ranks > 1 ? peer(sums, 0) : sums)->band >= kInf;
  scale_stretch(t, lo, hi, lane, f, zero);
  if (ranks > 1) cluster_barrier();  // (the first CTA stays until it has been read)
}

// ---------------------------------------------------------------- AdamW

constexpr int kAdamThreads = 256, kAdamCtas = 3;  // CTAs an SM

__device__ __forceinline__ void load8(const void* p, int64_t e, bool bf16, float (&x)[8]) {
  if (bf16) {
    const uint4 r = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + e));
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) x[2 * j] = bf16lo(w[j]), x[2 * j + 1] = bf16hi(w[j]);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 r = __ldcs(reinterpret_cast<const float4*>(static_cast<const float*>(p) + e + 4 * h));
      x[4 * h] = r.x, x[4 * h + 1] = r.y, x[4 * h + 2] = r.z, x[4 * h + 3] = r.w;
    }
  }
}
__device__ __forceinline__ void store8(void* p, int64_t e, bool bf16, const float (&x)[8]) {
  if (bf16) {
    __stcs(reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + e),
           make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7])));
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      __stcs(reinterpret_cast<float4*>(static_cast<float*>(p) + e + 4 * h),
             make_float4(x[4 * h], x[4 * h + 1], x[4 * h + 2], x[4 * h + 3]));
  }
}
__device__ __forceinline__ float load1(const void* p, int64_t e, bool bf16) {
  return element(static_cast<const char*>(p), e, bf16 ? 2 : 4);
}
__device__ __forceinline__ void store1(void* p, int64_t e, bool bf16, float v) {
  store_element(static_cast<char*>(p), e, bf16 ? 2 : 4, v);
}

// A CTA a tile of 4096 elements: 16 a thread, all loads before the first store. Bound by HBM: 131 M parameters (bf16
// with fp32 masters, 28 bytes each) with their norm 576 us, 1.01 of the copy bandwidth; 29 M fp32 in 203 uneven tensors
// 116 us in the kernel, 7.0 TB/s. (Persistent CTAs 671 us for the first, tiles of 2048 595, 8 elements a thread 675.)
struct AdamStep {
  AdamRates r;
  float factor;
  bool skip;
  __device__ __forceinline__ void operator()(float g, float& w, float& m, float& v) const {
    if (skip) return;
    g *= factor;
    m = fmaf(r.beta1, m, r.rest1 * g);
    v = fmaf(r.beta2, v, r.rest2 * (g * g));
    w = fmaf(w, r.keep, -(r.rate * m) / fmaf(sqrtf(v), r.inv_root, r.eps));
  }
};

__device__ __forceinline__ void adam_one(const AdamEntry& e, int64_t x, const AdamStep& step) {
  float w = load1(e.w, x, e.w_bf16), m = e.m[x], v = e.v[x];
  step(load1(e.g, x, e.g_bf16), w, m, v);
  e.m_out[x] = m;
  e.v_out[x] = v;
  store1(e.w_out, x, e.w_bf16, w);
  if (e.p_out != nullptr) store1(e.p_out, x, e.p_bf16, w);
}

// 1 - beta^t from log beta, to 2^-23 of itself or so.
__device__ __forceinline__ float one_less_power(int64_t t, float log_hi, float log_low) {
  if (log_hi == -INFINITY) return 1.0f;
  const float hi = float(t), low = float(t - int64_t(hi)), p = hi * log_hi;
  const float rest = fmaf(hi, log_hi, -p) + (hi * log_low + low * log_hi), e = expm1f(p);
  return -(e + rest * (1.0f + e));
}

template <int CAP>
__global__ void __launch_bounds__(kAdamThreads, kAdamCtas) adamw_kernel(const __grid_constant__ AdamTable<CAP> t, AdamJob job) {
  grid_dependency_wait();
  grid_dependents_launch();
  AdamStep step = {job.rates, job.grad_scale, false};
  if (job.device_step != nullptr || job.device_lr != nullptr) {
    // In fp32 by one thread. 131 M elements, bf16 with masters: 518 us, as with the host's rates (517); in fp64 663;
    // in fp32 by every thread 543, and the spills that this brings take the host's to 521.
    __shared__ float rate, inv_root, keep;
    if (threadIdx.x == 0) {
      const int64_t steps = job.device_step != nullptr ? max(*job.device_step, int64_t(1)) : job.step;
      const float lr = job.device_lr != nullptr ? *job.device_lr : job.lr;
      rate = lr / one_less_power(steps, job.log1, job.log1_low);
      inv_root = 1.0f / sqrtf(one_less_power(steps, job.log2, job.log2_low));
      keep = fmaf(-lr, job.weight_decay, 1.0f);
    }
    __syncthreads();
    step.r.rate = rate;
    step.r.inv_root = inv_root;
    step.r.keep = keep;
  }
  if (job.clip != nullptr) {
    step.factor = job.clip[1] * job.grad_scale;
    step.skip = job.clip[3] == 0.0f;
    if (step.skip && job.in_place) return;
  }
  const int tile = blockIdx.x;
  const int at = entry_of(t, tile, threadIdx.x % 32);
  const AdamEntry& e = t.e[at];
  const int64_t from = int64_t(tile - e.first) * kAdamTile;
  if (e.phase == 255) {
    const int64_t to = min(e.count, from + kAdamTile);
    for (int64_t x = from + threadIdx.x; x < to; x += kAdamThreads) adam_one(e, x, step);
    return;
  }
  // groups of 8 elements at multiples of 8 in memory
  constexpr int kGroups = kAdamTile / (8 * kAdamThreads);
  const int64_t x0 = from + 8 * int(threadIdx.x) - e.phase;
  if (x0 >= 0 && x0 + 8 * kAdamThreads * (kGroups - 1) + 8 <= e.count) {
    float g[kGroups][8], w[kGroups][8], m[kGroups][8], v[kGroups][8];
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      const int64_t x = x0 + 8 * kAdamThreads * i;
      load8(e.g, x, e.g_bf16, g[i]);
      load8(e.w, x, e.w_bf16, w[i]);
      load8(e.m, x, false, m[i]);
      load8(e.v, x, false, v[i]);
    }
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      const int64_t x = x0 + 8 * kAdamThreads * i;
#pragma unroll
      for (int j = 0; j < 8; ++j) step(g[i][j], w[i][j], m[i][j], v[i][j]);
      store8(e.m_out, x, false, m[i]);
      store8(e.v_out, x, false, v[i]);
      store8(e.w_out, x, e.w_bf16, w[i]);
      if (e.p_out != nullptr) store8(e.p_out, x, e.p_bf16, w[i]);
    }
    return;
  }
#pragma unroll 1
  for (int i = 0; i < kGroups; ++i) {
    const int64_t x = x0 + 8 * kAdamThreads * i;
    if (x >= 0 && x + 8 <= e.count) {
      float g[8], w[8], m[8], v[8];
      load8(e.g, x, e.g_bf16, g);
      load8(e.w, x, e.w_bf16, w);
      load8(e.m, x, false, m);
      load8(e.v, x, false, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) step(g[j], w[j], m[j], v[j]);
      store8(e.m_out, x, false, m);
      store8(e.v_out, x, false, v);
      store8(e.w_out, x, e.w_bf16, w);
      if (e.p_out != nullptr) store8(e.p_out, x, e.p_bf16, w);
    } else {
      for (int64_t y = max(x, int64_t(0)); y < min(x + 8, e.count); ++y) adam_one(e, y, step);
    }
  }
}

// ---------------------------------------------------------------- launches

// Launched so that it may be scheduled while the kernel before it drains; every
// kernel here waits for that one before it touches memory.
template <class... Params, class... Args>
cudaError_t launch(void (*kernel)(Params...), int64_t grid, int threads, int cluster, size_t smem, cudaStream_t stream,
                   const Args&... args) {
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
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

int64_t granules_of(const GradTensor& t) {
  const int64_t es = t.bf16 ? 2 : 4, off = int64_t(reinterpret_cast<uintptr_t>(t.in) & 15);
  return t.count == 0 ? 0 : (off + t.count * es + 15) / 16;
}

template <int CAP>
void fill(GradTable<CAP>& t, const GradTensor* g, int n) {
  t.n = n;
  t.granules = 0;
  for (int i = 0; i < n; ++i) {
    t.e[i] = {g[i].in, g[i].out, t.granules, g[i].count * 2 + (g[i].bf16 ? 1 : 0)};
    if (g[i].count > 0) t.granules += granules_of(g[i]) + kTensorGranules;
  }
}

// CTAs for a list: every warp has at least 2 granules a lane, every SM two CTAs.
int64_t norm_ctas(int64_t granules) {
  const int64_t warps = kNormThreads / 32, most = std::min<int64_t>(2 * device_sms(), kMaxGradCtas);
  return std::max<int64_t>(1, std::min<int64_t>(most, (granules + warps * 64 - 1) / (warps * 64)));
}

// Granules a warp that the norm keeps in the L2 for the scaling.
int64_t granules_kept(int64_t per, int64_t ctas) { return std::min(per, kKept / 16 / (ctas * (kNormThreads / 32))); }

template <int CAP>
cudaError_t launch_norm_group(const GradTensor* g, int n, bool clip, const GradJob& job, int group, int groups, cudaStream_t stream) {
  GradTable<CAP> t;
  fill(t, g, n);
  const int64_t ctas = norm_ctas(t.granules);
  t.per = stretch(t.granules, ctas * (kNormThreads / 32));
  const bool max = job.kind == AR_NORM_MAX;
  cudaError_t err = cudaSuccess;
  // (of a longer list, the last launch's: the first to be scaled)
  t.keep = clip && group == groups - 1 ? granules_kept(t.per, ctas) : 0;
  if (t.granules > 0)
    err = launch(t.keep > 0 ? (max ? norm_kernel<CAP, true, true> : norm_kernel<CAP, false, true>)
                            : (max ? norm_kernel<CAP, true, false> : norm_kernel<CAP, false, false>),
                 ctas, kNormThreads, 1, 0, stream, t, job);
  if (err != cudaSuccess) return err;
  return launch(max ? finish_kernel<CAP, true> : finish_kernel<CAP, false>, 1, 1024, 1, sizeof(Value) * size_t(ctas + n), stream,
                t, job, group, groups);
}

template <int CAP>
cudaError_t launch_scale_group(const GradTensor* g, int n, bool last, const GradJob& job, cudaStream_t stream) {
  GradTable<CAP> t;
  fill(t, g, n);
  if (t.granules == 0) return cudaSuccess;
  const int64_t ctas = norm_ctas(t.granules);
  t.per = stretch(t.granules, ctas * (kNormThreads / 32));
  t.keep = last ? granules_kept(t.per, ctas) : 0;
  return launch(scale_kernel<CAP>, ctas, kNormThreads, 1, 0, stream, t, job);
}

// Lists of at most this many granules (1.5 MB for a norm, 0.5 MB for clipping) take one launch. Measured, one launch
// against two or three (us in a graph of calls, bf16, one tensor and 20 tensors): norm of 0.25 MB 5.1 / 6.3 and
// 5.8 / 8.4, 1 MB 6.3 / 6.7 and 7.4 / 8.7, 2 MB 7.3 / 6.6 and 9.1 / 8.5; clipping of 0.25 MB 8.5 / 8.6 and 9.5 / 12.0,
// 0.5 MB 10.1 / 8.7 and 11.9 / 12.1, 1 MB 12.2 / 9.0 and 14.0 / 12.2.
constexpr int64_t kShortNorm = 3 << 15, kShortClip = 1 << 15;

cudaError_t launch_short(GradTable<kGradCapSmall>& t, bool clip, const GradJob& job, cudaStream_t stream) {
  int ranks = 1;  // 4 granules a lane, where there are as many
  while (ranks < kMaxRanks && t.granules > int64_t(ranks) * kNormThreads * 4) ranks *= 2;
  t.keep = 0;
  t.per = std::max<int64_t>(32, stretch(t.granules, ranks * (kNormThreads / 32)));
  const bool max = job.kind == AR_NORM_MAX;
  return launch(clip ? (max ? short_kernel<true, true> : short_kernel<false, true>)
                     : (max ? short_kernel<true, false> : short_kernel<false, false>),
                ranks, kNormThreads, ranks, 0, stream, t, job);
}

template <int CAP>
cudaError_t launch_adam_group(const AdamEntry* e, int n, const AdamJob& job, cudaStream_t stream) {
  AdamTable<CAP> t;
  t.n = n;
  int64_t tiles = 0;
  for (int i = 0; i < n; ++i) {
    t.e[i] = e[i];
    t.e[i].first = int32_t(tiles);
    if (e[i].count > 0) tiles += (e[i].count + (e[i].phase == 255 ? 0 : e[i].phase) + kAdamTile - 1) / kAdamTile;
  }
  if (tiles == 0) return cudaSuccess;
  if (tiles > INT32_MAX) return cudaErrorInvalidConfiguration;
  t.tiles = int(tiles);
  return launch(adamw_kernel<CAP>, tiles, kAdamThreads, 1, 0, stream, t, job);
}

}  // namespace

cudaError_t launch_grad_norm(const GradTensor* g, int n, bool clip, const GradJob& job, cudaStream_t stream) {
  if (n <= kGradCapSmall) {
    GradTable<kGradCapSmall> t;
    fill(t, g, n);
    if (t.granules <= (clip ? kShortClip : kShortNorm)) return launch_short(t, clip, job, stream);
  }
  const int groups = (n + kGradCap - 1) / kGradCap;
  cudaError_t err = cudaSuccess;
  for (int k = 0; k < groups && err == cudaSuccess; ++k) {
    const int from = k * kGradCap, m = std::min(kGradCap, n - from);
    GradJob part = job;
    if (job.norms != nullptr) part.norms = job.norms + from;
    err = n <= kGradCapSmall ? launch_norm_group<kGradCapSmall>(g, n, clip, part, 0, 1, stream)
                             : launch_norm_group<kGradCap>(g + from, m, clip, part, k, groups, stream);
  }
  for (int k = groups - 1; clip && k >= 0 && err == cudaSuccess; --k) {
    const int from = k * kGradCap, m = std::min(kGradCap, n - from);
    err = n <= kGradCapSmall ? launch_scale_group<kGradCapSmall>(g, n, true, job, stream)
                             : launch_scale_group<kGradCap>(g + from, m, k == groups - 1, job, stream);
  }
  return err;
}

cudaError_t launch_adamw(const AdamEntry* e, int n, const AdamJob& job, cudaStream_t stream) {
  cudaError_t err = cudaSuccess;
  for (int from = 0; from < n && err == cudaSuccess; from += kAdamCap)
    err = n <= kAdamCapSmall ? launch_adam_group<kAdamCapSmall>(e, n, job, stream)
                             : launch_adam_group<kAdamCap>(e + from, std::min(kAdamCap, n - from), job, stream);
  return err;
}

}  // namespace ar
