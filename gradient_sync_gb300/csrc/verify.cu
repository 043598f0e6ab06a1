// Verification of drafted tokens against the target's probabilities (speculative
// sampling: Leviathan et al. 2023, Chen et al. 2023).
//
// For a row of target logits x, p_i = w_i / Z with
//   w_i = 2^(x_i k - c), k = log2(e) / temperature, Z = sum w_i,
// for any integer c (sums with other shifts join without rounding), and alike q
// for the draft's row. The draft t of the row stands while u < p_t / q_t. Where it
// falls, a token is drawn from max(p_i - q_i, 0), that is from w_i - v_i (Z / Z')
// where positive (v, Z' the draft's): the first index whose running sum passes u
// times the total.
//
//  sums_kernel  Z and Z' of every row, in parts of a row, a CTA each: one pass, no CTA waits
//               for another. Where a call has more rows than run at once, they are visited by
//               their place in their sequence; the last CTA of a row to finish decides about
//               its draft, and rows behind one that fell are not read any more.
//  draw_kernel  a cluster of up to 8 CTAs a sequence: joins the parts, finds the first draft
//               that falls, draws from that row alone (read two or three times, from the L2
//               where it is still there), writes the tokens.
// Results do not depend on which rows were skipped: none up to the first fall is.
//
// A draw has to put u on the right side of borders that may lie anywhere, also between
// tokens of 1e-6 and less. Its terms are fp32 exponentials, as in the sums: each is off by some
// 2^-22 of itself, and by half a last place of its exponent x k - c. Sums beyond 64 terms, and
// borders, are pairs of fp32 numbers; the draft's weight is subtracted in one fused operation.
//
// What bounds it, one GB300, calls in a graph: 64 sequences of 8 drafts x 131072 bf16, a third of the
// drafts standing, 47.4 us for the 149 MB of 285 that are not skipped and a draw: latency; 68 us where
// all stand and all is read. By themselves, caches cold: sums 38.8 us (3.9 TB/s; 56.3 us, 5.1 TB/s, where all
// is read), draw 19 us, half of it instructions fetched for the first time. One sequence of 4 drafts
// x 32000 fp32: 10.3 us, two kernels, latency. Draft rows at another alignment than the target's are
// read by elements (contiguous rows of 131073 tokens 85 us for 48), and threads whose scores are all masked go
// through their groups twice (all but 50 tokens of a row at -inf: 70 us for 48).
// Taken apart and left: rows held in shared memory by clusters that decide and draw
// themselves (99 us for the batch: barriers of a cluster take 0.6 us each, five a row, and
// rows that fall in vain are drawn from); fp64 for borders (an operation takes a warp some 200
// cycles: 16 us for the one sequence); weights to fp32's last place (draws 46 us for 27).
#include "verify.h"

#include <algorithm>

#include "common.cuh"
#include "pairs.cuh"

namespace ar {
namespace {

constexpr int kRowThreads = 256, kRowWarps = kRowThreads / 32;
constexpr int kMaxRanks = 8;  // CTAs of a cluster of draw_kernel

enum Mode : int { kLookup = 0, kDrafted = 1, kGreedy = 2 };  // drafts without distributions, with them, greedy

__device__ __forceinline__ Pair exp2_pair(Pair a) {
  const float2 y = floats_of(a);
  return pair_of(exp2_approx(y.x), exp2_approx(y.y));
}

__device__ __forceinline__ bool above(Two a, Two b) {
  const Two d = add(a, {-b.hi, -b.lo});
  return d.hi > 0.0f || (d.hi == 0.0f && d.lo > 0.0f);
}
__device__ __forceinline__ Two times(Two a, float u) {
  const float p = a.hi * u;
  return two_sum(p, fmaf(a.hi, u, -p) + a.lo * u);
}
__device__ __forceinline__ Two shuffled(Two v, int from) {
  return {__shfl_sync(~0u, v.hi, from), __shfl_sync(~0u, v.lo, from)};
}
__device__ __forceinline__ Two warp_sum(Two v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = add(v, {__shfl_xor_sync(~0u, v.hi, o), __shfl_xor_sync(~0u, v.lo, o)});
  return v;
}

// ---------------------------------------------------------------- rows

// A row of scores, in groups of 8 that start on 16 aligned bytes of the target's row.
template <bool BF16>
struct Scores {
  static constexpr int ES = BF16 ? 2 : 4, W = 16 / ES;
  static constexpr int kVecs = 8 / W;  // 16-byte vectors of a group
  const char* row;
  int n;
  int lead;      // elements between 16 aligned bytes and the first one
  bool aligned;  // groups start on 16 aligned bytes of this row too
  float bias;    // taken off every score: 0, or the maximum where scores are so large that x k has no fraction
  __device__ __forceinline__ Scores(const VerifyRows& r, int at, int64_t vocab) {
    row = r.data + int64_t(at) * r.ld * ES;
    n = int(vocab);
    lead = int(reinterpret_cast<uintptr_t>(row) / ES & (W - 1));
    aligned = true;
    bias = 0.0f;
  }
  __device__ __forceinline__ float one(int i) const {
    return BF16 ? bf16_to_f32(reinterpret_cast<const uint16_t*>(row)[i]) : reinterpret_cast<const float*>(row)[i];
  }
  // The group at element i as it lies in memory; -inf for elements outside the row.
  __device__ __forceinline__ void fetch(int i, uint4 (&r)[kVecs]) const {
    if (aligned && i >= 0 && i + 8 <= n) {
#pragma unroll
      for (int h = 0; h < kVecs; ++h) r[h] = __ldg(reinterpret_cast<const uint4*>(row + int64_t(i) * ES) + h);
    } else {
      edge(i, r);
    }
  }
  __device__ __forceinline__ void edge(int i, uint4 (&r)[kVecs]) const {
    uint32_t w[4 * kVecs];
#pragma unroll
    for (int j = 0; j < 4 * kVecs; ++j) w[j] = BF16 ? 0xFF80FF80u : 0xFF800000u;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (i + j < 0 || i + j >= n) continue;
      if (BF16) w[j / 2] = (w[j / 2] & (j % 2 ? 0x0000FFFFu : 0xFFFF0000u)) | uint32_t(reinterpret_cast<const uint16_t*>(row)[i + j]) << (16 * (j % 2));
      else w[j % (4 * kVecs)] = reinterpret_cast<const uint32_t*>(row)[i + j];
    }
#pragma unroll
    for (int h = 0; h < kVecs; ++h) r[h] = make_uint4(w[4 * h], w[4 * h + 1], w[4 * h + 2], w[4 * h + 3]);
  }
  static __device__ __forceinline__ void nothing(uint4 (&r)[kVecs]) {
    const uint32_t w = BF16 ? 0xFF80FF80u : 0xFF800000u;
#pragma unroll
    for (int h = 0; h < kVecs; ++h) r[h] = make_uint4(w, w, w, w);
  }
  // Its scores, less the bias.
  __device__ __forceinline__ void scores(const uint4 (&r)[kVecs], float (&x)[8]) const {
#pragma unroll
    for (int h = 0; h < kVecs; ++h) {
      const uint32_t w[4] = {r[h].x, r[h].y, r[h].z, r[h].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (BF16) x[2 * j] = bf16lo(w[j]), x[(2 * j + 1) % 8] = bf16hi(w[j]);
        else x[4 * h + j] = __uint_as_float(w[j]);
      }
    }
    if (bias != 0.0f) {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] -= bias;
    }
  }
  __device__ __forceinline__ void load(int i, float (&x)[8]) const {
    uint4 r[kVecs];
    fetch(i, r);
    scores(r, x);
  }
};

// Groups of 8 elements: element 8 g + first is group g's first.
struct Piece {
  int lo, hi, first;
};

// ---------------------------------------------------------------- sums

// 2^d for d <= 0, exactly (0 below the normal numbers).
__device__ __forceinline__ float pow2(int d) { return d > -127 ? __int_as_float((d + 127) << 23) : 0.0f; }

// A sum s * 2^c. kNone: of nothing but -inf (s = 0). kLow: of scores so low that x k
// has no fraction (beside any others they are nothing). At kOdd, above all shifts, s = +inf: of scores
// so high. s is NaN where a score was NaN or +inf.
struct Sum {
  int c;
  float s;
};
constexpr int kNone = -(1 << 28), kLow = -(1 << 27), kOdd = 1 << 28;
constexpr float kFraction = 4194304.0f;  // 2^22
__device__ __forceinline__ Sum normalized(int c, float s) {  // s a normal number: to [1/2, 1)
  const int bits = __float_as_int(s);
  return {c + (bits >> 23) - 126, __int_as_float((bits & 0x007fffff) | 0x3f000000)};
}
// The sum over a warp's lanes.
__device__ __forceinline__ Sum warp_join(Sum v) {
  const int c = __reduce_max_sync(~0u, v.c);
  float s = v.s * pow2(v.c - c);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
  return {c, s};
}

struct Top {
  float x;
  int at;
};
__device__ __forceinline__ Top larger(Top a, Top b) { return b.x > a.x || (b.x == a.x && b.at < a.at) ? b : a; }
__device__ __forceinline__ Top largest(Top v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = larger(v, {__shfl_xor_sync(~0u, v.x, o), __shfl_xor_sync(~0u, v.at, o)});
  return v;
}
__device__ __forceinline__ float max8(const float (&x)[8]) {
  return fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
}

// Sums that the first group's shift does not serve: with the thread's maximum.
template <class S>
__device__ __noinline__ Sum careful_sum(const S s, const Piece p, int start, int step, float k) {
  float top = -INFINITY, x[8];
  bool nan = false;
  for (int g = p.lo + start; g < p.hi; g += step) {
    s.load(8 * g + p.first, x);
    for (int j = 0; j < 8; ++j) top = fmaxf(top, x[j]), nan |= x[j] != x[j];
  }
  if (nan || top == INFINITY) return {0, __int_as_float(0x7fc00000)};
  if (top == -INFINITY) return {kNone, 0.0f};
  if (top * k >= kFraction) return {kOdd, INFINITY};
  if (top * k <= -kFraction) return {kLow, 0.5f};
  const float c = ceilf(top * k);
  Two sum = {0.0f, 0.0f};
  for (int g = p.lo + start; g < p.hi; g += step) {
    s.load(8 * g + p.first, x);
    float t = 0.0f;
    for (int j = 0; j < 8; ++j) t += exp2_approx(fmaf(x[j], k, -c));
    sum = add(sum, {t, 0.0f});
  }
  return normalized(int(c), sum.hi);
}

// The sum over every step-th group from the start-th, in one pass: the shift is the first group's. Scores far above it
// have exponents of up to 100, of which fp32 leaves 2^-18. (A batch taken again with its own maximum as the shift:
// 64 x 8 drafts x 131072 bf16 49.8 us for 48.1, at a temperature of 0.2 55 for 44.) TOP: and the largest score with its
// first place.
template <bool TOP, class S>
__device__ __forceinline__ Sum fast_sum(const S& s, const Piece& p, int start, int step, float k, Top& top) {
  constexpr int kDeep = 8 / S::kVecs;  // groups of 8 loads in flight
  int g = p.lo + start;
  if (TOP) top = {-INFINITY, INT32_MAX};
  if (g >= p.hi) return {kNone, 0.0f};
  float c = 0.0f;
  const Pair kk = pair_of(k, k);
  Pair cc = kk;
  int best = g;
  bool begun = false;
  Two sum = {0.0f, 0.0f};
#pragma unroll 1
  for (; g < p.hi; g += kDeep * step) {
    uint4 raw[kDeep][S::kVecs];
#pragma unroll
    for (int r = 0; r < kDeep; ++r) {
      S::nothing(raw[r]);
      if (g + r * step < p.hi) s.fetch(8 * (g + r * step) + p.first, raw[r]);
    }
    if (!begun) {
      float x[8];
      s.scores(raw[0], x);
      const float m = max8(x);
      c = fabsf(m * k) < kFraction ? ceilf(m * k) : 0.0f;
      cc = pair_of(-c, -c);
      begun = true;
    }
    Pair a = pair_of(0.0f, 0.0f), b = a;
#pragma unroll
    for (int r = 0; r < kDeep; ++r) {
      float x[8];
      s.scores(raw[r], x);
      if (TOP) {
        const float m = max8(x);
        if (m > top.x) top.x = m, best = g + r * step;
      }
#pragma unroll
      for (int j = 0; j < 8; j += 4) {
        a = add2(a, exp2_pair(fma2(pair_of(x[j], x[j + 1]), kk, cc)));
        b = add2(b, exp2_pair(fma2(pair_of(x[j + 2], x[j + 3]), kk, cc)));
      }
    }
    const float2 v = floats_of(add2(a, b));
    sum = add(sum, {v.x + v.y, 0.0f});
  }
  if (TOP) {
    float y[8];
    s.load(8 * best + p.first, y);
#pragma unroll
    for (int j = 7; j >= 0; --j)
      if (y[j] == top.x) top.at = 8 * best + p.first + j;
  }
  // A term that the shift was taken from is above 1/2: less is the sum behind a first group of masked scores, whose
  // terms may be below fp32's range.
  if (sum.hi > 0.25f && sum.hi < 1.2e30f) return normalized(int(c), sum.hi);
  return careful_sum(s, p, start, step, k);
}

// ---------------------------------------------------------------- decisions

// log2 of a sum, in two parts.
__device__ __forceinline__ Two log2_of(Sum v) { return two_sum(float(v.c), log2f(v.s)); }
// x k less such a logarithm, in two parts. (k as the sum has it, without what fp32 leaves of it.)
__device__ __forceinline__ Two log2_p(float x, float k, Two log2_z) {
  const float p = x * k;
  return add(two_sum(p, -log2_z.hi), {fmaf(x, k, -p) - log2_z.lo, 0.0f});
}
__device__ __forceinline__ float to_e(Two v) {  // times log 2
  return fmaf(v.hi, 0.693147182f, fmaf(v.hi, -1.90465421e-9f, v.lo * 0.693147182f));
}

// What a warp or CTA tells others: two numbers of two rows.
struct alignas(16) Post {
  float a, b, c, d;
};
__device__ __forceinline__ Post post_of(float4 v) { return {v.x, v.y, v.z, v.w}; }

// A place in a sequence: its row of the target, and where the sequence is.
struct Place {
  int row, s, first, count, j;
  __device__ __forceinline__ bool behind() const { return j == count; }  // the row behind all drafts
};

struct Verdict {
  int stands;  // 1: the draft stands; 0: it falls, or there is none; -1: a row is no distribution; 2: scores are odd
  float logp;  // of the draft that stands; greedy: of the largest
  int best;    // greedy
  Sum zx, zy;
  float bias_x, bias_y;
};

__device__ __forceinline__ int start_of(const VerifyParams& p, int64_t s) {
  if (p.draft_start == nullptr) return s == 0 ? 0 : int(p.n_drafts);
  return int(min(max(p.draft_start[s], int64_t(0)), p.n_drafts));
}

// A row's sum with its maximum taken off, by one warp.
template <class S>
__device__ __noinline__ Sum odd_sum(S s, float k, int lane, float& bias) {
  const Piece p = {0, (s.lead + s.n + 7) / 8, -s.lead};
  float top = -INFINITY;
  for (int g = lane; g < p.hi; g += 32) {
    float x[8];
    s.load(8 * g + p.first, x);
    top = fmaxf(top, max8(x));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
  s.bias = bias = top;
  return warp_join(careful_sum(s, p, lane, 32, k));
}

// One warp's verdict on a draft from the parts of its rows' sums. ODD: scores too high or low are worked out
// here (slowly, from the rows); else such a row has no verdict.
template <bool XB, bool YB, int MODE, bool ODD>
__device__ __forceinline__ Verdict decide(const VerifyParams& p, const Place& at, int lane) {
  const bool drafted = MODE == kDrafted && !at.behind();
  Scores<XB> x(p.target, at.row, p.vocab);
  Scores<YB> y(drafted ? p.draft : p.target, drafted ? at.first + at.j : at.row, p.vocab);
  // (these loads are independent of the parts')
  const int64_t token = at.behind() ? -1 : p.drafts[at.first + at.j];
  float u = 0.0f, xt = -INFINITY, yt = -INFINITY;
  if (MODE != kGreedy && token >= 0 && token < p.vocab) {
    u = p.uniforms[at.row];
    xt = x.one(int(token));
    if (drafted) yt = y.one(int(token));
  }
  Post v = {__int_as_float(kNone), 0.0f, MODE == kGreedy ? -INFINITY : __int_as_float(kNone), MODE == kGreedy ? __int_as_float(INT32_MAX) : 0.0f};
  if (lane < p.parts) v = post_of(__ldcg(reinterpret_cast<const float4*>(p.sums + int64_t(at.row) * p.parts + lane)));
  Sum zx = warp_join({__float_as_int(v.a), v.b}), zy = {0, 0.5f};
  Top top = {v.c, __float_as_int(v.d)};
  if (MODE == kGreedy) top = largest(top);
  if (drafted) zy = warp_join({__float_as_int(v.c), v.d});
  Verdict r = {-1, 0.0f, top.at, {0, 0.5f}, {0, 0.5f}, 0.0f, 0.0f};
  if (zx.s == INFINITY || zx.c == kLow || zy.s == INFINITY || zy.c == kLow) {
    if (!ODD) {
      r.stands = 2;
      return r;
    }
    if (zx.s == INFINITY || zx.c == kLow) zx = odd_sum(x, p.target.k, lane, r.bias_x);
    if (drafted && (zy.s == INFINITY || zy.c == kLow)) zy = odd_sum(y, p.draft.k, lane, r.bias_y);
  }
  // neither NaN nor nothing
  if (!(zx.s > 0.0f && zx.s < INFINITY && zy.s > 0.0f && zy.s < INFINITY)) return r;
  r.zx = zx = normalized(zx.c, zx.s);
  r.zy = zy = normalized(zy.c, zy.s);
  const Two log2_zx = log2_of(zx);
  r.stands = 0;
  if (MODE == kGreedy) {
    r.stands = !at.behind() && token == top.at;
    r.logp = to_e(log2_p(top.x - r.bias_x, p.target.k, log2_zx));
    return r;
  }
  if (!(xt > -INFINITY)) return r;
  const Two lp = log2_p(xt - r.bias_x, p.target.k, log2_zx);
  Two gap = lp;
  if (drafted) {
    const Two lq = log2_p(yt - r.bias_y, p.draft.k, log2_of(zy));
    gap = add(lp, {-lq.hi, -lq.lo});
  }
  // (a draft that its own distribution gives nothing stands; a NaN falls)
  if (u == u && (u <= 0.0f || (drafted && yt == -INFINITY) ||
                 fminf(u, 0.99999994f) < exp2f(gap.hi) * fmaf(gap.lo, 0.69314718f, 1.0f)))
    r.stands = 1;
  r.logp = to_e(lp);
  return r;
}

template <bool XB, bool YB, int MODE>
__global__ void __launch_bounds__(kRowThreads, 4) sums_kernel(const __grid_constant__ VerifyParams p) {
  grid_dependency_wait();
  grid_dependents_launch();
  __shared__ Post posts[kRowWarps];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int part = int(blockIdx.x) & (p.parts - 1);
  const int64_t row = int64_t(blockIdx.x >> p.part_bits) * p.pitch + blockIdx.y;
  if (row >= p.n_drafts + p.n_seq) return;
  // the row's sequence: the last one whose first row is not behind this one, found among as many as there are threads
  // at a time
  int seq = 0;
  for (int64_t end = p.n_seq;;) {
    const int64_t step = (end - seq + kRowThreads - 1) / kRowThreads, i = seq + threadIdx.x * step;
    const int n = __syncthreads_count(i < end && start_of(p, i) + i <= row);
    if (n == 0) return;
    seq += int((n - 1) * step);
    if (step == 1) break;
    end = min(end, seq + step);
  }
  const int first = start_of(p, seq), count = max(start_of(p, seq + 1) - first, 0);
  const Place at = {int(row), seq, first, count, int(row) - first - seq};
  if (at.j < 0 || at.j > count) return;
  if (p.fallen != nullptr && at.j > 0 &&
      __syncthreads_or(threadIdx.x == 0 && *const_cast<volatile int*>(p.fallen + seq) < at.j))
    return;
  const bool drafted = MODE == kDrafted && !at.behind();
  const Scores<XB> x(p.target, at.row, p.vocab);
  Scores<YB> y(drafted ? p.draft : p.target, drafted ? at.first + at.j : at.row, p.vocab);
  y.aligned = ((y.lead - x.lead) & (y.W - 1)) == 0;
  // this CTA's part, in groups that start on 16 aligned bytes of the target's row
  const int groups = int((x.lead + p.vocab + 7) / 8), per = (groups + p.parts - 1) >> p.part_bits;
  const Piece piece = {min(groups, part * per), min(groups, (part + 1) * per), -x.lead};
  // half of the warps for each row, where there are two
  constexpr int kHalf = kRowWarps / 2;
  Top top, none;
  Sum z;
  if (!drafted) z = fast_sum<MODE == kGreedy>(x, piece, threadIdx.x, kRowThreads, p.target.k, top);
  else if (warp < kHalf) z = fast_sum<false>(x, piece, threadIdx.x, 32 * kHalf, p.target.k, none);
  else z = fast_sum<false>(y, piece, threadIdx.x - 32 * kHalf, 32 * kHalf, p.draft.k, none);
  z = warp_join(z);
  if (MODE == kGreedy) top = largest(top);
  if (lane == 0) posts[warp] = {__int_as_float(z.c), z.s, MODE == kGreedy ? top.x : 0.0f, MODE == kGreedy ? __int_as_float(top.at) : 0.0f};
  __syncthreads();
  if (warp != 0) return;
  const Post v = posts[lane % kRowWarps];
  z = {__float_as_int(v.a), v.b};
  const Sum nothing = {kNone, 0.0f};
  Sum zx = warp_join(lane < (drafted ? kHalf : kRowWarps) ? z : nothing), zy = nothing;
  if (drafted) zy = warp_join(lane >= kHalf && lane < kRowWarps ? z : nothing);
  if (MODE == kGreedy) top = largest({v.c, __float_as_int(v.d)});
  // (sums of many parts grow by a factor of 32 a level: to [1/2, 1) again)
  if (zx.s > 0.0f && zx.s < INFINITY && zx.c > kLow) zx = normalized(zx.c, zx.s);
  if (zy.s > 0.0f && zy.s < INFINITY && zy.c > kLow) zy = normalized(zy.c, zy.s);
  int last = 0;
  if (lane == 0) {
    __stcg(reinterpret_cast<float4*>(p.sums + int64_t(at.row) * p.parts + part),
           MODE == kGreedy ? make_float4(__int_as_float(zx.c), zx.s, top.x, __int_as_float(top.at))
                           : make_float4(__int_as_float(zx.c), zx.s, __int_as_float(zy.c), zy.s));
    if (p.fallen != nullptr) {
      __threadfence();
      last = atomicAdd(p.done + at.row, 1) == p.parts - 1;
    }
  }
  if (p.fallen == nullptr || at.behind() || !__shfl_sync(~0u, last, 0)) return;
  __threadfence();
  const Verdict r = decide<XB, YB, MODE, false>(p, at, lane);
  if (lane == 0 && (r.stands == 0 || r.stands == -1)) atomicMin(p.fallen + at.s, at.j);
}

// ---------------------------------------------------------------- draws

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ Two peer_post(const Two* p, int rank) {
  Two v;
  asm volatile(
      "{\n"
      ".reg .b32 remote;\n"
      "mapa.shared::cluster.u32 remote, %2, %3;\n"
      "ld.shared::cluster.v2.f32 {%0, %1}, [remote];\n"
      "}\n"
      : "=f"(v.hi), "=f"(v.lo)
      : "r"(uint32_t(__cvta_generic_to_shared(p))), "r"(rank)
      : "memory");
  return v;
}

// 2^(x k - c), two at a time.
struct Weights {
  Pair k, minus_c;
  __device__ __forceinline__ Weights(const VerifyRows& r, int shift)
      : k(pair_of(r.k, r.k)), minus_c(pair_of(-float(shift), -float(shift))) {}
  __device__ __forceinline__ Pair of(float x0, float x1) const { return exp2_pair(fma2(pair_of(x0, x1), k, minus_c)); }
};

__device__ __forceinline__ Pair sum4(const Pair (&w)[4]) { return add2(add2(w[0], w[1]), add2(w[2], w[3])); }

// What a token is drawn from: w_i, less the draft's weight (a row's, or one token's).
enum Less : int { kNothing = 0, kRow = 1, kToken = 2 };
template <class X, class Y>
struct Draw {
  X x;
  Y y;
  Weights wx, wy;
  float rho, rho_low;  // Z / Z'
  int token;
  int less;
  // A group's weights.
  __device__ __forceinline__ void weights(const uint4 (&rx)[X::kVecs], const uint4 (&ry)[Y::kVecs], int i, Pair (&w)[4]) const {
    float a[8];
    x.scores(rx, a);
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = wx.of(a[2 * j], a[2 * j + 1]);
    if (less == kRow) {
      y.scores(ry, a);
      const Pair r = pair_of(-rho, -rho), r_low = pair_of(-rho_low, -rho_low);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const Pair v = wy.of(a[2 * j], a[2 * j + 1]);
        const float2 d = floats_of(fma2(v, r_low, fma2(v, r, w[j])));
        w[j] = pair_of(fmaxf(d.x, 0.0f), fmaxf(d.y, 0.0f));
      }
    } else if (less == kToken) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 d = floats_of(w[j]);
        w[j] = pair_of(i + 2 * j == token ? 0.0f : d.x, i + 2 * j + 1 == token ? 0.0f : d.y);
      }
    }
  }
  __device__ __forceinline__ void fetch(int i, uint4 (&rx)[X::kVecs], uint4 (&ry)[Y::kVecs]) const {
    x.fetch(i, rx);
    if (less == kRow) y.fetch(i, ry);
  }
  // The weight of a lane's groups.
  __device__ __forceinline__ Two total(const Piece& p, int lane) const {
    constexpr int kRounds = 4 / (X::kVecs > Y::kVecs ? X::kVecs : Y::kVecs);  // loaded together
    Two sum = {0.0f, 0.0f};
#pragma unroll 1
    for (int g = p.lo + lane; g < p.hi; g += kRounds * 32) {
      uint4 rx[kRounds][X::kVecs], ry[kRounds][Y::kVecs];
#pragma unroll
      for (int r = 0; r < kRounds; ++r) {
        X::nothing(rx[r]);
        Y::nothing(ry[r]);
        if (g + 32 * r < p.hi) fetch(8 * (g + 32 * r) + p.first, rx[r], ry[r]);
      }
      Pair a = pair_of(0.0f, 0.0f);
#pragma unroll
      for (int r = 0; r < kRounds; ++r) {
        Pair w[4];
        weights(rx[r], ry[r], 8 * (g + 32 * r) + p.first, w);
        a = add2(a, sum4(w));
      }
      const float2 f = floats_of(a);
      sum = add(sum, {f.x + f.y, 0.0f});
    }
    return sum;
  }
};

// Of parts one behind the other, two a lane, behind a sum of `before`: the part that the border lies in, and the sum
// before it. Behind the last border by rounding: the last part with weight; -1: none has any.
struct Border {
  int part;
  Two before;
};
__device__ __forceinline__ Border border_of(Two v0, Two v1, Two before, Two target, int lane) {
  Two run = add(v0, v1);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Two v = {__shfl_up_sync(~0u, run.hi, o), __shfl_up_sync(~0u, run.lo, o)};
    if (lane >= o) run = add(run, v);
  }
  // (a lane's sum before its parts is the one of the lanes before, rounded alike for both)
  Two mine = {__shfl_up_sync(~0u, run.hi, 1), __shfl_up_sync(~0u, run.lo, 1)};
  mine = lane > 0 ? add(before, mine) : before;
  const Two middle = add(mine, v0);
  const bool first = v0.hi > 0.0f && above(middle, target), second = v1.hi > 0.0f && above(add(before, run), target);
  const unsigned over = __ballot_sync(~0u, first || second), some = __ballot_sync(~0u, v0.hi > 0.0f || v1.hi > 0.0f);
  if (some == 0) return {-1, before};
  const int owner = over != 0 ? __ffs(int(over)) - 1 : 31 - __clz(int(some));
  const bool low = over != 0 ? first : !(v1.hi > 0.0f);
  return {2 * owner + (__shfl_sync(~0u, int(low), owner) != 0 ? 0 : 1), shuffled(low ? mine : middle, owner)};
}

struct Shared {
  Two posts[2][kRowWarps];
  Verdict verdicts[kRowWarps];
  Border border;  // of a draw: its part is rank * kRowWarps + warp
  Two target;
  Two parts[kRowWarps];
};

// CTAS: of them an SM.
template <bool XB, bool YB, int MODE, int CTAS>
__global__ void __launch_bounds__(kRowThreads, CTAS) draw_kernel(const __grid_constant__ VerifyParams p) {
  using X = Scores<XB>;
  using Y = Scores<YB>;
  grid_dependency_wait();
  grid_dependents_launch();
  __shared__ Shared sh;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int ranks = 1 << p.rank_bits, rank = int(blockIdx.x) & (ranks - 1), s = int(blockIdx.x >> p.rank_bits);
  const int first = start_of(p, s), count = max(start_of(p, s + 1) - first, 0), row0 = first + s;
  // a warp a draft, eight at a time, until one falls (there is none in the last row); where rows may have been skipped
  // it is the one that they were skipped for, and those behind it have no sums
  const int stop = p.fallen != nullptr ? __ldcg(p.fallen + s) : INT32_MAX;
  int a;
  for (int j0 = 0;; j0 += kRowWarps) {
    const int j = j0 + warp;
    Verdict v = {0};
    if (j <= min(count, stop)) {
      v = decide<XB, YB, MODE, true>(p, {row0 + j, s, first, count, j}, lane);
      if (j == stop) v.stands = min(v.stands, 0);
      if (lane == 0) sh.verdicts[warp] = v;
    }
    __syncthreads();
    a = j0;
    while (a < j0 + kRowWarps && a < count && sh.verdicts[a - j0].stands == 1) ++a;
    if (rank == 0 && lane == 0 && j < a) {
      p.tokens[row0 + j] = p.drafts[first + j];
      p.logp[row0 + j] = v.logp;
    }
    if (a < j0 + kRowWarps) break;
    __syncthreads();
  }
  const Verdict at = sh.verdicts[a % kRowWarps];
  if (rank == 0) {
    if (threadIdx.x == 0) p.accepted[s] = a;
    for (int j = a + 1 + int(threadIdx.x); j <= count; j += kRowThreads) {
      p.tokens[row0 + j] = -1;
      p.logp[row0 + j] = 0.0f;
    }
  }
  const int row = row0 + a;
  if (MODE == kGreedy || at.stands < 0) {
    if (rank == 0 && threadIdx.x == 0) {
      p.tokens[row] = at.stands < 0 || at.best < 0 || at.best >= p.vocab ? -1 : at.best;
      p.logp[row] = at.stands < 0 ? __int_as_float(0x7fc00000) : at.logp;
    }
    return;
  }

  const bool behind = a == count, drafted = MODE == kDrafted && !behind;
  X x(p.target, row, p.vocab);
  Y y(drafted ? p.draft : p.target, drafted ? first + a : row, p.vocab);
  y.aligned = ((y.lead - x.lead) & (Y::W - 1)) == 0;
  // this CTA's part, in groups that start on 16 aligned bytes of the target's row, and its warps' (whole rounds):
  // indexes order like (rank, warp, round, lane, element)
  const int groups = int((x.lead + p.vocab + 7) / 8), per = (groups + ranks - 1) >> p.rank_bits;
  const int g0 = min(groups, rank * per), g1 = min(groups, g0 + per);
  const int per_warp = (g1 - g0 + 32 * kRowWarps - 1) / (32 * kRowWarps) * 32;
  const auto piece_of = [&](int w) { return Piece{min(g1, g0 + w * per_warp), min(g1, g0 + (w + 1) * per_warp), -x.lead}; };
  const Piece piece = piece_of(warp);
  const int64_t token = behind || drafted ? -1 : p.drafts[first + a];
  const float last = p.uniforms[row0 + count];
  const float u = fminf(fmaxf(last == last ? last : 0.0f, 0.0f), 0.99999994f);
  Draw<X, Y> d = {x, y, Weights(p.target, at.zx.c), Weights(drafted ? p.draft : p.target, at.zy.c), 0.0f, 0.0f,
                  token >= 0 && token < p.vocab ? int(token) : -1, behind ? kNothing : drafted ? kRow : kToken};
  d.x.bias = at.bias_x;
  d.y.bias = at.bias_y;
  const float v_bias = at.bias_x;
  const Sum v_zx = at.zx;
  if (drafted) {  // the quotient of the sums: rounded, and what that leaves
    d.rho = at.zx.s / at.zy.s;
    d.rho_low = fmaf(-d.rho, at.zy.s, at.zx.s) / at.zy.s;
  }

  // the total of what is drawn from (once more of p itself, where there is no residue), and the piece that the border
  // lies in
  Border border;
  Two target;
#pragma unroll 1
  for (int again = 0;; ++again) {
    const Two sum = warp_sum(d.total(piece, lane));
    if (lane == 0) sh.posts[again][warp] = sum;
    // posts are written once, then read by every CTA's first warp, two a lane
    if (ranks > 1) cluster_barrier();
    else __syncthreads();
    if (warp == 0) {
      Two v[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = 2 * lane + h;
        v[h] = {0.0f, 0.0f};
        if (i < ranks * kRowWarps)
          v[h] = ranks > 1 ? peer_post(&sh.posts[again][i % kRowWarps], i / kRowWarps) : sh.posts[again][i];
      }
      target = times(warp_sum(add(v[0], v[1])), u);
      border = border_of(v[0], v[1], {0.0f, 0.0f}, target, lane);
      if (lane == 0) sh.border = border, sh.target = target;
    }
    __syncthreads();
    border = sh.border;
    target = sh.target;
    if (border.part >= 0 || again > 0) break;
    d.less = kNothing;
  }
  if (ranks > 1) asm volatile("barrier.cluster.arrive.release;" ::: "memory");  // (this CTA reads no other's posts any more)

  if (border.part >= 0 && border.part / kRowWarps == rank) {
    // the piece, split over all warps again and again, until a lane has one group
    Piece q = piece_of(border.part % kRowWarps);
#pragma unroll 1
    for (;;) {
      const int per_part = ((q.hi - q.lo + kRowWarps - 1) / kRowWarps + 31) / 32 * 32;
      const Piece part = {min(q.hi, q.lo + warp * per_part), min(q.hi, q.lo + (warp + 1) * per_part), q.first};
      Pair w[4];
      Two mine;
      if (per_part == 32) {
        uint4 rx[X::kVecs], ry[Y::kVecs];
        X::nothing(rx);
        Y::nothing(ry);
        if (part.lo + lane < part.hi) d.fetch(8 * (part.lo + lane) + q.first, rx, ry);
        d.weights(rx, ry, 8 * (part.lo + lane) + q.first, w);
        const float2 f = floats_of(sum4(w));
        mine = {f.x + f.y, 0.0f};
      } else {
        mine = d.total(part, lane);
      }
      const Two sum = warp_sum(mine);
      if (lane == 0) sh.parts[warp] = sum;
      __syncthreads();
      const Border at = border_of(lane < kRowWarps ? sh.parts[lane % kRowWarps] : Two{0.0f, 0.0f}, {0.0f, 0.0f}, border.before, target, lane);
      if (per_part > 32) {
        border.before = at.before;
        q = {min(q.hi, q.lo + at.part / 2 * per_part), min(q.hi, q.lo + (at.part / 2 + 1) * per_part), q.first};
        __syncthreads();
        continue;
      }
      if (at.part / 2 == warp) {
        const Border in = border_of(mine, {0.0f, 0.0f}, at.before, target, lane);
        if (lane == in.part / 2) {  // (never -1: the warp's sum is not 0)
          const int i = 8 * (part.lo + lane) + q.first;
          Two run = in.before;
          int hit = -1, last = -1;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 f = floats_of(w[j / 2]);
            const float v = j % 2 ? f.y : f.x;
            run = add(run, {v, 0.0f});
            if (v > 0.0f) {
              last = i + j;
              if (hit < 0 && above(run, target)) hit = last;
            }
          }
          const int found = hit >= 0 ? hit : last;
          p.tokens[row] = found;
          p.logp[row] = found >= 0 ? to_e(log2_p(x.one(found) - v_bias, p.target.k, log2_of(v_zx))) : 0.0f;
        }
      }
      break;
    }
  }
  if (ranks > 1) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");  // no CTA goes while another may still read from it
}

// No row is done, and no draft of any sequence has fallen yet.
__global__ void __launch_bounds__(256) clear_kernel(const __grid_constant__ VerifyParams p) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i < p.n_seq) p.fallen[i] = INT32_MAX;
  if (i < p.n_drafts + p.n_seq) p.done[i] = 0;
}

// ---------------------------------------------------------------- launches

// Launched so that it may be scheduled while the kernel before it drains; every
// kernel here waits for that one before it touches memory.
cudaError_t launch_after(void (*kernel)(VerifyParams), const VerifyParams& p, dim3 grid, int cluster, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kRowThreads);
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

using Kernel = void (*)(VerifyParams);

Kernel sums_of(const VerifyParams& p) {
  const bool x = p.target.bf16 != 0, y = p.draft.bf16 != 0;
  if (p.greedy) return x ? sums_kernel<true, true, kGreedy> : sums_kernel<false, false, kGreedy>;
  if (p.draft.data == nullptr) return x ? sums_kernel<true, true, kLookup> : sums_kernel<false, false, kLookup>;
  if (x) return y ? sums_kernel<true, true, kDrafted> : sums_kernel<true, false, kDrafted>;
  return y ? sums_kernel<false, true, kDrafted> : sums_kernel<false, false, kDrafted>;
}
template <int CTAS>
Kernel draw_of(const VerifyParams& p) {
  const bool x = p.target.bf16 != 0, y = p.draft.bf16 != 0;
  if (p.draft.data == nullptr) return x ? draw_kernel<true, true, kLookup, CTAS> : draw_kernel<false, false, kLookup, CTAS>;
  if (x) return y ? draw_kernel<true, true, kDrafted, CTAS> : draw_kernel<true, false, kDrafted, CTAS>;
  return y ? draw_kernel<false, true, kDrafted, CTAS> : draw_kernel<false, false, kDrafted, CTAS>;
}

// Elements that a CTA of sums_kernel takes, of one row or two. Measured, 16384 of each of two rows against 8192 and
// 32768: 64 x 8 drafts x 131072 bf16 54.5, 58.2 and 58.4 us. At least 4096 where there are few rows, against 8192: one
// sequence of 4 drafts x 32000 fp32 10.4 and 12.2 us, 8 of 8 drafts 12.0 and 13.4.
constexpr int64_t kPart = 32768, kLeastPart = 4096;
// ... of draw_kernel: a round of all its warps. (Clusters of 8 against 4: 4 x 4 drafts x 131072 bf16 13.5 and 16.9 us.)
constexpr int64_t kLeastDraw = 2048;
// Calls with less to read do not skip rows, which takes about 3 us: flags cleared by a launch, rows decided about.
// Measured, skipping against not: 64 x 8 drafts x 131072 bf16 (285 MB) 50 and 64 us, 256 x 4 x 32000 (147 MB) 41.8 and
// 43.3, 16 x 4 x 131072 (38 MB) 20.1 and 18.2, 200 x 3 looked-up drafts x 5000 (8 MB) 16.6 and 13.3.
constexpr int64_t kSkipBytes = int64_t(96) << 20;

}  // namespace

cudaError_t launch_verify(const VerifyParams& q, cudaStream_t stream) {
  VerifyParams p = q;
  const int64_t rows = p.n_drafts + p.n_seq, sms = device_sms();
  // parts of a row: of a good size, or smaller where that keeps SMs without work
  p.part_bits = 0;
  const int64_t part = p.draft.data != nullptr ? kPart / 2 : kPart;
  while (p.part_bits < kVerifyPartBits && (p.vocab >> p.part_bits) > part) ++p.part_bits;
  while (p.part_bits < kVerifyPartBits && (rows << p.part_bits) < 2 * sms && (p.vocab >> p.part_bits) >= 2 * kLeastPart) ++p.part_bits;
  while (p.part_bits > 0 && (rows << p.part_bits) > 0x7fffffff) --p.part_bits;
  p.parts = 1 << p.part_bits;
  // more rows than run at once, and enough of them: by their place in their sequence, and not behind a draft that fell
  const int64_t bytes = p.vocab * (rows * (p.target.bf16 ? 2 : 4) + (p.draft.data == nullptr ? 0 : p.n_drafts * (p.draft.bf16 ? 2 : 4)));
  const bool waves = rows * p.parts > 4 * sms && bytes > kSkipBytes && p.n_drafts > 0 && rows / p.n_seq < 60000;
  p.pitch = waves ? int((rows + p.n_seq - 1) / p.n_seq) : 1;
  if (!waves) p.fallen = nullptr;
  // a cluster a sequence, all at once where they fit: three CTAs an SM, or, with fewer registers, four where that makes
  // the clusters larger (64 x 8 drafts x 131072 bf16 48.0 us with four, 50.8 with three; where it does not, 16 x 8 x 32000
  // 14.5 and 13.6)
  const auto rank_bits = [&](int64_t ctas) {
    int bits = 0;
    while ((1 << bits) < kMaxRanks && (p.n_seq << bits) * 2 <= ctas * sms && (p.vocab >> bits) >= 2 * kLeastDraw) ++bits;
    return bits;
  };
  p.rank_bits = p.greedy ? 0 : rank_bits(3);
  Kernel draw = p.target.bf16 ? draw_kernel<true, true, kGreedy, 4> : draw_kernel<false, false, kGreedy, 4>;
  if (!p.greedy) {
    const bool more = rank_bits(4) > p.rank_bits;
    if (more) p.rank_bits = rank_bits(4);
    draw = more ? draw_of<4>(p) : draw_of<3>(p);
  }
  cudaError_t err = cudaSuccess;
  if (err == cudaSuccess && waves) err = launch_after(clear_kernel, p, dim3(unsigned((rows + 255) / 256)), 1, stream);
  const int64_t across = (rows + p.pitch - 1) / p.pitch;
  if (err == cudaSuccess)
    err = launch_after(sums_of(p), p, dim3(unsigned(across << p.part_bits), unsigned(p.pitch)), 1, stream);
  if (err == cudaSuccess)
    err = launch_after(draw, p, dim3(unsigned(p.n_seq << p.rank_bits)), 1 << p.rank_bits, stream);
  return err;
}

}  // namespace ar
