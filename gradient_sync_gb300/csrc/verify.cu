// Verification of drafted tokens against the target's probabilities.
//
// For a row of target logits x, p_i = w_i / Z with
//   w_i = 2^(x_i k - c), k = log2(e) / temperature, Z = sum w_i,
// for any integer c (sums with other shifts join without rounding), and alike q
// for the draft's row. The draft t of the row stands while
// u < p_t / q_t. Where it falls, a token is drawn from max(p_i - q_i, 0),
// that is from w_i - v_i (Z / Z') where positive (v, Z' the draft's): the first index whose
// running sum passes u times the total.
//
// rows_kernel: a cluster of up to 8 CTAs takes a row of the target with its row of
// the draft, copies both to shared memory, and works from there: sums, decision,
// and, where the draft falls, the draw. Each row is read from HBM once; rows
// too long for eight SMs' shared memory are read again by every pass. The rows of a sequence
// run side by side, and each leaves what the sequence would need of it (stands or
// not, the token drawn, both log-probabilities). Rows behind a draft that fell are
// not needed: where a call has more rows than run at once, rows are visited by
// their place in their sequence, and one that starts after such a fall is skipped.
// tokens_kernel, a warp a sequence, finds the first draft that falls and writes
// the tokens. Results do not depend on which rows were skipped.
//
// A draw has to put u on the right side of borders that may lie anywhere, also
// between tokens of 1e-6 and less. So its weights are to fp32's last place (the
// fast ones of the sums that only decide about drafts are not): the exponent is
// carried with what fp32 leaves of it, the draft's weight is subtracted in one fused operation with a two-part factor, and sums
// are pairs of fp32 numbers (fp64 adds are slow here), borders 64 bits.
#include "verify.h"

#include <algorithm>

#include "bulk.cuh"
#include "common.cuh"

namespace ar {
namespace {

constexpr int kRowThreads = 256, kRowWarps = kRowThreads / 32;
constexpr int kMaxRanks = 8;  // CTAs of a cluster

enum Mode : int { kLookup = 0, kDrafted = 1, kGreedy = 2 };  // drafts without distributions, with them, greedy

constexpr uint32_t kPolls = 1u << 22;  // of a copy, each of which may suspend the thread for a while

extern __shared__ __align__(16) char held[];

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
__device__ __forceinline__ Pair exp2_pair(Pair a) {
  const float2 y = floats_of(a);
  return pair_of(exp2_approx(y.x), exp2_approx(y.y));
}

// A sum as two fp32 numbers: about 46 bits.
struct Two {
  float hi, lo;
};
__device__ __forceinline__ Two two_sum(float a, float b) {
  const float s = a + b, z = s - a;
  return {s, (a - (s - z)) + (b - z)};
}
__device__ __forceinline__ Two add(Two a, Two b) {
  Two s = two_sum(a.hi, b.hi);
  const float lo = s.lo + (a.lo + b.lo);
  const float hi = s.hi + lo;
  return {hi, lo - (hi - s.hi)};
}
__device__ __forceinline__ double wide(Two a) { return double(a.hi) + double(a.lo); }
__device__ __forceinline__ Two warp_sum(Two v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = add(v, {__shfl_xor_sync(~0u, v.hi, o), __shfl_xor_sync(~0u, v.lo, o)});
  return v;
}

// What every warp of a cluster tells the others in one phase.
struct alignas(16) Post {
  float a, b, c, d;
};
enum Phase : int { kSums = 0, kTops = 1, kSumsAgain = 2, kExact = 3, kTotals = 4, kTotalsAgain = 5, kPhases = 6 };

// A sum s * 2^c.
struct Sum {
  int c;
  float s;
};

struct Shared {
  Post posts[kPhases][kRowWarps];
  uint64_t full[kRowWarps];  // a warp's part of the rows is in shared memory
  int abort;
  int skip;
  int odd;    // scores so large that their bias has to be taken off first: 1: the target's, 2: the draft's
  int stands;
  float bias_x, bias_y;
  Sum zx, zy;
  float rho, rho_low;
  int owner;  // of a draw's border: rank * kRowWarps + warp, -1: no weight
  double before, target;
  Two parts[kRowWarps];
  Two log2_z;
};

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ Post peer_post(const Post* p, int rank) {
  Post v;
  asm volatile(
      "{\n"
      ".reg .b32 remote;\n"
      "mapa.shared::cluster.u32 remote, %4, %5;\n"
      "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [remote];\n"
      "}\n"
      : "=f"(v.a), "=f"(v.b), "=f"(v.c), "=f"(v.d)
      : "r"(uint32_t(__cvta_generic_to_shared(p))), "r"(rank)
      : "memory");
  return v;
}
__device__ __forceinline__ int peer_int(const int* p, int rank) {
  int v;
  asm volatile(
      "{\n"
      ".reg .b32 remote;\n"
      "mapa.shared::cluster.u32 remote, %1, %2;\n"
      "ld.shared::cluster.s32 %0, [remote];\n"
      "}\n"
      : "=r"(v)
      : "r"(uint32_t(__cvta_generic_to_shared(p))), "r"(rank)
      : "memory");
  return v;
}

// A phase's posts are written once, then read by every CTA's first warp, two a lane.
__device__ __forceinline__ void posted(int ranks) {
  if (ranks > 1) cluster_barrier();
  else __syncthreads();
}
__device__ __forceinline__ Post post_at(const Shared& sh, int phase, int i, int ranks) {
  const Post* p = &sh.posts[phase][i % kRowWarps];
  return ranks > 1 ? peer_post(p, i / kRowWarps) : *p;
}

// A row of scores as a warp sees it: its part in shared memory, where it has
// been copied to, or the row itself.
template <bool BF16, bool HOLD>
struct Scores {
  static constexpr int ES = BF16 ? 2 : 4, W = 16 / ES;
  const char* row;
  int n;
  int lead;      // elements between 16 aligned bytes and the first one
  int shift;     // HOLD: element i is at held + shift + i * ES
  bool aligned;  // groups of 8 start on 16 aligned bytes
  float bias;    // taken off every score: 0, or the maximum where scores are so large that x k has no fraction
  __device__ Scores(const VerifyRows& r, int64_t at, int64_t vocab) {
    row = r.data + at * r.ld * ES;
    n = int(vocab);
    lead = int(reinterpret_cast<uintptr_t>(row) / ES % W);
    shift = 0;
    aligned = true;
    bias = 0.0f;
  }
  __device__ __forceinline__ void place(int from, int offset) { shift = offset - (from - (from + lead + 8) % W) * ES; }
  // Copies the elements [from, to) to where place() has put them, -inf for those that the row does not have: whole 16
  // aligned bytes by one bulk copy (its size is returned), the others by the lanes. (from >= -7)
  __device__ uint32_t copy(int from, int to, int lane, uint64_t* bar) const {
    const int head = lead > 0 ? W - lead : 0, tail = max(head, (lead + n) / W * W - lead);
    const int a = max(from - (from + lead + 8) % W, head), b = min(to + (W - (to + lead) % W) % W, tail);
    const int few = lane < W ? (lane < head ? lane : -1) : tail + lane - W;  // edges: elements 0 .. head - 1, tail .. n - 1
    if (lane < 2 * W && few >= max(from, 0) && few < min(to, n)) put(few, one(few));
    if (lane < 8 && from + lane < 0) put(from + lane, -INFINITY);
    if (lane < 8 && to - 1 - lane >= n) put(to - 1 - lane, -INFINITY);
    if (b <= a) return 0;
    if (lane == 0) bulk_load(held + shift + a * ES, row + int64_t(a) * ES, uint32_t(b - a) * ES, bar);
    return uint32_t(b - a) * ES;
  }
  __device__ __forceinline__ void put(int i, float x) const {
    if (BF16) *reinterpret_cast<uint16_t*>(held + shift + i * ES) = uint16_t(__float_as_uint(x) >> 16);
    else *reinterpret_cast<float*>(held + shift + i * ES) = x;
  }
  __device__ __forceinline__ const char* at(int i) const { return HOLD ? held + shift + i * ES : row + int64_t(i) * ES; }
  __device__ __forceinline__ float one(int i) const {  // from the row
    return BF16 ? bf16_to_f32(reinterpret_cast<const uint16_t*>(row)[i]) : reinterpret_cast<const float*>(row)[i];
  }
  // Elements i .. i + 7; -inf for those outside the row.
  __device__ __forceinline__ void load(int i, float (&x)[8]) const {
    load_as_is(i, x);
    if (bias != 0.0f) {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] -= bias;
    }
  }
  __device__ __forceinline__ void load_as_is(int i, float (&x)[8]) const {
    if (aligned && (HOLD || (i >= 0 && i + 8 <= n))) {
      if (BF16) {
        const uint4 r = *reinterpret_cast<const uint4*>(at(i));
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) x[2 * j] = bf16lo(w[j]), x[2 * j + 1] = bf16hi(w[j]);
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float4 r = reinterpret_cast<const float4*>(at(i))[h];
          x[4 * h] = r.x, x[4 * h + 1] = r.y, x[4 * h + 2] = r.z, x[4 * h + 3] = r.w;
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x[j] = -INFINITY;
        if (HOLD || (i + j >= 0 && i + j < n))
          x[j] = BF16 ? bf16_to_f32(*reinterpret_cast<const uint16_t*>(at(i + j))) : *reinterpret_cast<const float*>(at(i + j));
      }
    }
  }
};

// The groups of 8 elements of a warp: element 8 g + first is group g's first. A
// warp's groups lie one behind the other, so that indexes order like (rank,
// warp, round, lane, element).
struct Piece {
  int lo, hi, first;
};

// The largest score of a warp's piece, and its first place.
template <class S>
__device__ __forceinline__ float top_of(const S& s, const Piece& p, int lane) {
  float top = -INFINITY;
#pragma unroll 2
  for (int g = p.lo + lane; g < p.hi; g += 32) {
    float x[8];
    s.load_as_is(8 * g + p.first, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) top = fmaxf(top, x[j]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
  return top;
}

// 2^d for d <= 0, exactly (0 below the normal numbers).
__device__ __forceinline__ float pow2(int d) { return d > -127 ? __int_as_float((d + 127) << 23) : 0.0f; }

// Sums: kNone for a part that is all -inf (s = 0). s is NaN where a score was NaN
// or +inf, +inf (at kOdd, above all shifts) where a bias has to be taken off first.
constexpr int kNone = -(1 << 28), kOdd = 1 << 28;
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

// Sums that the first group's shift does not serve: with the thread's maximum.
template <class S>
__device__ __noinline__ Sum careful_sum(const S s, const Piece p, int lane, float k) {
  float top = -INFINITY, sum = 0.0f, x[8];
  bool nan = false;
  for (int g = p.lo + lane; g < p.hi; g += 32) {
    s.load(8 * g + p.first, x);
    for (int j = 0; j < 8; ++j) top = fmaxf(top, x[j]), nan |= x[j] != x[j];
  }
  if (nan || top == INFINITY) return {0, __int_as_float(0x7fc00000)};
  if (top == -INFINITY) return {kNone, 0.0f};
  if (!(fabsf(top * k) < 4194304.0f)) return {kOdd, INFINITY};
  const float c = ceilf(top * k);
  for (int g = p.lo + lane; g < p.hi; g += 32) {
    s.load(8 * g + p.first, x);
    for (int j = 0; j < 8; ++j) sum += exp2_approx(fmaf(x[j], k, -c));
  }
  return normalized(int(c), sum);
}

// The sum over a thread's groups, in one pass: the shift is the first group's. TOP: and the largest score with
// its first place.
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
__device__ __forceinline__ Sum joined(Sum a, Sum b) {
  const int c = max(a.c, b.c);
  return {c, a.s * pow2(a.c - c) + b.s * pow2(b.c - c)};
}
template <bool TOP, class S>
__device__ __forceinline__ Sum fast_sum(const S& s, const Piece& p, int lane, float k, Top& top) {
  int g = p.lo + lane;
  if (TOP) top = {-INFINITY, INT32_MAX};
  if (g >= p.hi) return {kNone, 0.0f};
  float x[8];
  s.load(8 * g + p.first, x);
  float m = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
  const float c = fabsf(m * k) < 4194304.0f ? ceilf(m * k) : 0.0f;
  const Pair kk = pair_of(k, k), cc = pair_of(-c, -c);
  int best = g;
  if (TOP) top.x = m;
  Two sum = {0.0f, 0.0f};
  while (g < p.hi) {
    Pair a = pair_of(0.0f, 0.0f), b = a;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (g < p.hi) {
        s.load(8 * g + p.first, x);
        if (TOP) {
          m = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
          if (m > top.x) top.x = m, best = g;
        }
#pragma unroll
        for (int j = 0; j < 8; j += 4) {
          a = add2(a, exp2_pair(fma2(pair_of(x[j], x[j + 1]), kk, cc)));
          b = add2(b, exp2_pair(fma2(pair_of(x[j + 2], x[j + 3]), kk, cc)));
        }
      }
      g += 32;
    }
    const float2 v = floats_of(add2(a, b));
    sum = add(sum, {v.x + v.y, 0.0f});
  }
  if (TOP) {
    s.load(8 * best + p.first, x);
#pragma unroll
    for (int j = 7; j >= 0; --j)
      if (x[j] == top.x) top.at = 8 * best + p.first + j;
  }
  if (sum.hi > 7.9e-31f && sum.hi < 1.2e30f) return normalized(int(c), sum.hi);
  return careful_sum(s, p, lane, k);
}

// 2^(x k - c) to fp32's last place; 0 where it is below 2^-126.
struct Weight {
  float k, k_low, c;
  __device__ __forceinline__ float operator()(float x) const {
    const float p = fmaxf(x * k, c - 200.0f), t = p - c;  // (the limit: -inf has no differences)
    const float left = fmaf(x, k_low, fmaf(x, k, -p)) + (p - (t + c));
    const float e = exp2_approx(t);
    return t > -200.0f ? fmaf(e, left * 0.69314718f, e) : 0.0f;
  }
};

template <class S>
__device__ __forceinline__ Two exact_sum(const S& s, const Piece& p, int lane, const Weight& w) {
  Two sum = {0.0f, 0.0f};
#pragma unroll 2
  for (int g = p.lo + lane; g < p.hi; g += 32) {
    float x[8];
    s.load(8 * g + p.first, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = w(x[j]);
    sum = add(sum, {((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7])), 0.0f});
  }
  return sum;
}

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

// What a token is drawn from: w_i, less the draft's weight (a row's, or one token's).
enum Less : int { kNothing = 0, kRow = 1, kToken = 2 };
template <class X, class Y>
struct Draw {
  const X& x;
  const Y& y;
  Weight wx, wy;
  float rho, rho_low;  // Z / Z'
  int token;
  int less;
  __device__ __forceinline__ float weights(int i, float (&w)[8]) const {
    x.load(i, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = wx(w[j]);
    if (less == kRow) {
      float v[8];
      y.load(i, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float a = wy(v[j]);
        w[j] = fmaxf(fmaf(-a, rho_low, fmaf(-a, rho, w[j])), 0.0f);
      }
    } else if (less == kToken) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i + j == token) w[j] = 0.0f;
    }
    return ((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7]));
  }
  __device__ __forceinline__ Two total(const Piece& p, int lane) const {
    Two sum = {0.0f, 0.0f};
#pragma unroll 2
    for (int g = p.lo + lane; g < p.hi; g += 32) {
      float w[8];
      sum = add(sum, {weights(8 * g + p.first, w), 0.0f});
    }
    return warp_sum(sum);
  }
};

// Of up to 64 parts one behind the other (each lane's two), the one that the border lies in, and the sum before it
// (one warp). Behind the last border by rounding: the last part with weight; -1: none has any.
__device__ __forceinline__ int part_of(double v0, double v1, double before_all, double target, int lane, double& before) {
  double run = v0 + v1;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double v = __shfl_up_sync(~0u, run, o);
    if (lane >= o) run += v;
  }
  run += before_all;
  const double mine = run - (v0 + v1);
  const bool first = v0 > 0.0 && mine + v0 > target, second = v1 > 0.0 && run > target;
  const unsigned over = __ballot_sync(~0u, first || second), some = __ballot_sync(~0u, v0 > 0.0 || v1 > 0.0);
  if (some == 0) return -1;
  const int owner = over != 0 ? __ffs(int(over)) - 1 : 31 - __clz(int(some));
  const bool low = over != 0 ? first : !(v1 > 0.0);
  before = __shfl_sync(~0u, low ? mine : mine + v0, owner);
  return 2 * owner + (__shfl_sync(~0u, int(low), owner) != 0 ? 0 : 1);
}

// The border's token, by the warp whose piece it lies in.
template <class D>
__device__ __forceinline__ int token_at(const D& d, const Piece& p, int lane, double before, double target) {
  int last = -1, hit = -1;
  for (int g0 = p.lo; g0 < p.hi && hit < 0; g0 += 32) {
    const int i = 8 * (g0 + lane) + p.first;
    float w[8];
    double chunk = 0.0;
    if (g0 + lane < p.hi) chunk = double(d.weights(i, w));
    double run = chunk;  // of the lanes up to this one
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double v = __shfl_up_sync(~0u, run, o);
      if (lane >= o) run += v;
    }
    const unsigned over = __ballot_sync(~0u, chunk > 0.0 && before + run > target), some = __ballot_sync(~0u, chunk > 0.0);
    if (some != 0) {
      // the lane that holds the border, else the last one with weight
      const int owner = over != 0 ? __ffs(int(over)) - 1 : 31 - __clz(int(some));
      if (lane == owner) {
        double at = before + (run - chunk);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          at += double(w[j]);
          if (w[j] > 0.0f) {
            last = i + j;
            if (at > target && hit < 0) hit = last;
          }
        }
        if (over != 0 && hit < 0) hit = last;
      }
      last = __shfl_sync(~0u, last, owner);
      hit = __shfl_sync(~0u, hit, owner);
    }
    before += __shfl_sync(~0u, run, 31);
  }
  return hit >= 0 ? hit : last;
}

__device__ __forceinline__ int64_t start_of(const VerifyParams& p, int64_t s) {
  if (p.draft_start == nullptr) return s == 0 ? 0 : p.n_drafts;
  return min(max(p.draft_start[s], int64_t(0)), p.n_drafts);
}

template <bool XB, bool YB, int MODE, bool HOLD>
__global__ void __launch_bounds__(kRowThreads) rows_kernel(const __grid_constant__ VerifyParams p) {
  using X = Scores<XB, HOLD>;
  using Y = Scores<YB, HOLD>;
  grid_dependency_wait();
  grid_dependents_launch();
  __shared__ Shared sh;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int ranks = p.ranks, rank = int(blockIdx.x) % ranks;
  // rows are visited `pitch` apart, so that those of a sequence come one after the other
  const int64_t item = int64_t(blockIdx.x) / ranks, across = (p.n_drafts + p.n_seq + p.pitch - 1) / p.pitch;
  const int64_t row = item % across * p.pitch + item / across;
  if (row >= p.n_drafts + p.n_seq) return;
  if (HOLD && threadIdx.x < kRowWarps) mbar_init(&sh.full[threadIdx.x], 1);
  if (threadIdx.x == 0) sh.abort = 0;
  if (HOLD) mbar_init_fence();
  // the sequence: the last one whose first row is not behind this one
  int64_t s = -1;
  for (int64_t base = 0; base < p.n_seq; base += kRowThreads) {
    const int64_t i = base + threadIdx.x;
    const int n = __syncthreads_count(i < p.n_seq && start_of(p, i) + i <= row);
    s += n;
    if (n < kRowThreads) break;
  }
  if (s < 0) return;
  const int64_t first = start_of(p, s), count = max(start_of(p, s + 1) - first, int64_t(0)), place = row - s - first;
  if (place < 0 || place > count) return;
  if (p.fallen != nullptr) {
    // all CTAs of the cluster go by what the first one sees
    if (threadIdx.x == 0) sh.skip = *const_cast<volatile int*>(p.fallen + s) < place;
    int skip;
    if (ranks > 1) {
      cluster_barrier();
      skip = peer_int(&sh.skip, 0);
      if (skip) cluster_barrier();  // (read by all before the first one goes)
    } else {
      __syncthreads();
      skip = sh.skip;
    }
    if (skip) return;
  }
  const bool behind = place == count;  // the row behind all drafts
  const bool drafted = MODE == kDrafted && !behind;
  X x(p.target, row, p.vocab);
  Y y(drafted ? p.draft : p.target, drafted ? first + place : row, p.vocab);
  if (drafted) y.aligned = ((y.lead - x.lead) & (Y::W - 1)) == 0;
  // this CTA's part, in groups that start on 16 aligned bytes of the target's row, and its warps' (whole rounds)
  const int groups = int((x.lead + p.vocab + 7) / 8), per = (groups + ranks - 1) / ranks;
  const int g0 = min(groups, rank * per), g1 = min(groups, g0 + per);
  const int per_warp = (g1 - g0 + 32 * kRowWarps - 1) / (32 * kRowWarps) * 32;
  const auto piece_of = [&](int w) { return Piece{min(g1, g0 + w * per_warp), min(g1, g0 + (w + 1) * per_warp), -x.lead}; };
  const Piece piece = piece_of(warp);
  // shared memory: the target's part, then the draft's, each warp's with up to 16 bytes on both sides
  const auto place_rows = [&](int w) {
    const Piece q = piece_of(w);
    x.place(8 * q.lo + q.first, (q.lo - g0) * 8 * X::ES);
    if (drafted) y.place(8 * q.lo + q.first, (g1 - g0) * 8 * X::ES + (q.lo - g0) * 8 * Y::ES + w * 32);
  };
  if (HOLD) place_rows(warp);
  if (HOLD && piece.lo < piece.hi) {
    const int from = 8 * piece.lo + piece.first, to = 8 * piece.hi + piece.first;
    uint32_t bytes = x.copy(from, to, lane, &sh.full[warp]);
    if (drafted) bytes += y.copy(from, to, lane, &sh.full[warp]);
    if (lane == 0) mbar_arrive_expect_tx(&sh.full[warp], bytes);
  }
  // what thread 0 needs for the decision
  int64_t token = -1;
  float xt = -INFINITY, yt = -INFINITY, u_draft = 0.0f, u_draw = 0.0f;
  if (!behind && (threadIdx.x == 0 || MODE == kLookup)) token = p.drafts[first + place];
  const bool inside = token >= 0 && token < p.vocab;
  if (MODE != kGreedy) {
    u_draw = p.uniforms[s + first + count];
    if (threadIdx.x == 0 && inside) {
      xt = x.one(int(token));
      if (drafted) yt = y.one(int(token));
      u_draft = p.uniforms[row];
    }
  }
  bool copied = true;
  if (HOLD && piece.lo < piece.hi) {
    const StatusRef status = {p.status_word, p.status_host};
    copied = mbar_wait(&sh.full[warp], 0, kPolls, &sh.abort, status);
    __syncwarp();
  }

  // the sums, once more where the scores turn out to be too large as they are
  const float kx = p.target.k, ky = p.draft.k;
  for (int again = 0; again < 2; ++again) {
    Top top, none;
    Sum zx = warp_join(fast_sum<MODE == kGreedy>(x, piece, lane, kx, top)), zy = {0, 0.5f};
    if (drafted) zy = warp_join(fast_sum<false>(y, piece, lane, ky, none));
    if (MODE == kGreedy) top = largest(top);
    if (lane == 0)
      sh.posts[2 * again][warp] = MODE == kGreedy ? Post{__int_as_float(zx.c), zx.s, top.x, __int_as_float(top.at)}
                                                  : Post{__int_as_float(zx.c), zx.s, __int_as_float(zy.c), zy.s};
    posted(ranks);
    if (warp == 0) {
      Sum ax[2], ay[2];
      Top at[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = lane + 32 * h;
        ax[h] = ay[h] = {kNone, 0.0f};
        at[h] = {-INFINITY, INT32_MAX};
        if (i < ranks * kRowWarps) {
          const Post v = post_at(sh, 2 * again, i, ranks);
          ax[h] = {__float_as_int(v.a), v.b};
          if (MODE == kGreedy) at[h] = {v.c, __float_as_int(v.d)};
          else ay[h] = {__float_as_int(v.c), v.d};
        }
      }
      zx = warp_join(joined(ax[0], ax[1]));
      if (MODE == kDrafted) zy = warp_join(joined(ay[0], ay[1]));
      if (MODE == kGreedy) top = largest(larger(at[0], at[1]));
      const int odd = again > 0 ? 0 : (zx.s == INFINITY ? 1 : 0) | (drafted && zy.s == INFINITY ? 2 : 0);
      // neither NaN nor nothing
      const bool ok = zx.s > 0.0f && zx.s < INFINITY && (!drafted || (zy.s > 0.0f && zy.s < INFINITY));
      if (lane == 0) sh.odd = odd;
      if (lane == 0 && odd == 0) {
        RowResult* result = p.results + row;
        bool fell = true;
        sh.stands = 1;  // 1: no draw follows
        if (!ok) {
          if (rank == 0) *result = {-1, __int_as_float(0x7fc00000), 0.0f, 0, 0};
        } else {
          sh.zx = zx = normalized(zx.c, zx.s);
          const Two log2_zx = log2_of(zx);
          sh.log2_z = log2_zx;
          if (MODE == kGreedy) {
            const float lp = to_e(log2_p(top.x, kx, log2_zx));
            fell = token != top.at;
            if (rank == 0) *result = {top.at, lp, lp, int32_t(!behind && !fell), 0};
          } else {
            sh.stands = 0;
            if (drafted) sh.zy = zy = normalized(zy.c, zy.s);
            if (xt > -INFINITY) {
              const Two lp = log2_p(xt - x.bias, kx, log2_zx);
              Two gap = lp;
              if (drafted) {
                const Two lq = log2_p(yt - y.bias, ky, log2_of(zy));
                gap = add(lp, {-lq.hi, -lq.lo});
              }
              // (a draft that its own distribution gives nothing stands)
              const bool stands = u_draft <= 0.0f || (drafted && yt == -INFINITY) ||
                                  fminf(u_draft, 0.99999994f) < exp2f(gap.hi) * fmaf(gap.lo, 0.69314718f, 1.0f);
              if (stands && u_draft == u_draft) {
                sh.stands = 1;
                fell = false;
                if (rank == 0) *result = {-1, 0.0f, to_e(lp), 1, 0};
              }
            }
          }
        }
        if (p.fallen != nullptr && rank == 0 && !behind && fell) atomicMin(p.fallen + s, int(place));
      }
    }
    __syncthreads();
    if (sh.odd == 0) break;
    const float mx = top_of(x, piece, lane), my = drafted ? top_of(y, piece, lane) : 0.0f;
    if (lane == 0) sh.posts[kTops][warp] = {mx, my, 0.0f, 0.0f};
    posted(ranks);
    if (threadIdx.x == 0) {
      float bx = mx, by = my;
      for (int i = 0; i < ranks * kRowWarps; ++i) {
        const Post v = post_at(sh, kTops, i, ranks);
        bx = fmaxf(bx, v.a), by = fmaxf(by, v.b);
      }
      sh.bias_x = sh.odd & 1 ? bx : 0.0f;
      sh.bias_y = sh.odd & 2 ? by : 0.0f;
    }
    __syncthreads();
    x.bias = sh.bias_x;
    y.bias = sh.bias_y;
  }
  if (MODE != kGreedy && !sh.stands) {
    Draw<X, Y> d = {x, y, {kx, p.target.k_low, float(sh.zx.c)}, {ky, p.draft.k_low, drafted ? float(sh.zy.c) : 0.0f}, 0.0f, 0.0f,
                    inside ? int(token) : -1, behind ? kNothing : drafted ? kRow : kToken};
    if (drafted) {
      const Two a = warp_sum(exact_sum(x, piece, lane, d.wx)), b = warp_sum(exact_sum(y, piece, lane, d.wy));
      if (lane == 0) sh.posts[kExact][warp] = {a.hi, a.lo, b.hi, b.lo};
      posted(ranks);
      if (warp == 0) {
        Two c = {0.0f, 0.0f}, e = {0.0f, 0.0f};
        for (int i = lane; i < ranks * kRowWarps; i += 32) {
          const Post v = post_at(sh, kExact, i, ranks);
          c = add(c, {v.a, v.b});
          e = add(e, {v.c, v.d});
        }
        c = warp_sum(c);
        e = warp_sum(e);
        // the quotient of both pairs: a rounded one, and what it leaves
        const float rho = c.hi / e.hi;
        if (lane == 0) sh.rho = rho, sh.rho_low = ((fmaf(-rho, e.hi, c.hi) + c.lo) - rho * e.lo) / e.hi;
      }
      __syncthreads();
      d.rho = sh.rho;
      d.rho_low = sh.rho_low;
    }
    const float u = fminf(fmaxf(u_draw == u_draw ? u_draw : 0.0f, 0.0f), 0.99999994f);
    for (int again = 0; again < 2; ++again) {
      const Two total = d.total(piece, lane);
      if (lane == 0) sh.posts[kTotals + again][warp] = {total.hi, total.lo, 0.0f, 0.0f};
      posted(ranks);
      if (warp == 0) {
        double v[2] = {0.0, 0.0}, before = 0.0;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (2 * lane + h < ranks * kRowWarps) {
            const Post t = post_at(sh, kTotals + again, 2 * lane + h, ranks);
            v[h] = wide({t.a, t.b});
          }
        double all = v[0] + v[1];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(~0u, all, o);
        const double target = double(u) * all;
        const int owner = part_of(v[0], v[1], 0.0, target, lane, before);
        if (lane == 0) sh.owner = owner, sh.before = before, sh.target = target;
      }
      __syncthreads();
      if (sh.owner >= 0) break;
      d.less = kNothing;  // no residue: from p itself
    }
    if (sh.owner >= 0 && sh.owner / kRowWarps == rank) {
      // the owner's piece, once more over all warps, then the round of the warp that has the border
      const Piece q = piece_of(sh.owner % kRowWarps);
      if (HOLD) place_rows(sh.owner % kRowWarps);
      const int per_part = ((q.hi - q.lo + kRowWarps - 1) / kRowWarps + 31) / 32 * 32;
      const Piece part = {min(q.hi, q.lo + warp * per_part), min(q.hi, q.lo + (warp + 1) * per_part), q.first};
      const Two total = d.total(part, lane);
      if (lane == 0) sh.parts[warp] = total;
      __syncthreads();
      const double v = lane < kRowWarps ? wide(sh.parts[lane]) : 0.0;
      double before = 0.0;
      const int owner = part_of(v, 0.0, sh.before, sh.target, lane, before) / 2;
      if (owner == warp) {
        const int found = token_at(d, part, lane, before, sh.target);
        if (lane == 0 && found >= 0)
          p.results[row] = {found, to_e(log2_p(x.one(found) - x.bias, kx, sh.log2_z)), 0.0f, 0, 0};
      }
    }
  }
  if (!copied) {  // (recorded; the copy may still be under way, and shared memory has to stay until it is not)
    for (uint32_t i = 0; i < kPolls && !mbar_try_wait(&sh.full[warp], 0); ++i) {
    }
  }
  if (ranks > 1) cluster_barrier();  // no CTA goes while another may still read from it
}

// No draft of any sequence has fallen yet.
__global__ void __launch_bounds__(256) clear_kernel(const __grid_constant__ VerifyParams p) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t s = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (s < p.n_seq) p.fallen[s] = INT32_MAX;
}

// A warp a sequence: the first draft that falls, and the tokens up to it.
__global__ void __launch_bounds__(256) tokens_kernel(const __grid_constant__ VerifyParams p) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t s = int64_t(blockIdx.x) * 8 + threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  if (s >= p.n_seq) return;
  const int64_t first = start_of(p, s), count = max(start_of(p, s + 1) - first, int64_t(0)), row = first + s;
  int64_t a = count;
  for (int64_t j = 0; j < count; j += 32) {
    const unsigned falls = __ballot_sync(~0u, j + lane < count && p.results[row + j + lane].stands == 0);
    if (falls != 0) {
      a = j + __ffs(int(falls)) - 1;
      break;
    }
  }
  for (int64_t j = lane; j <= count; j += 32) {
    const RowResult& r = p.results[row + j];
    int64_t token = -1;
    float logp = 0.0f;
    if (j < a) {
      token = p.drafts[first + j];
      logp = r.draft_logp;
    } else if (j == a) {
      token = r.token >= 0 && r.token < p.vocab ? r.token : -1;
      logp = r.token_logp;
    }
    p.tokens[row + j] = token;
    p.logp[row + j] = logp;
  }
  if (lane == 0) p.accepted[s] = a;
}

// Launched so that it may be scheduled while the kernel before it drains; every
// kernel here waits for that one before it touches memory.
cudaError_t launch_after(void (*kernel)(VerifyParams), const VerifyParams& p, int64_t grid, int threads, int cluster,
                         size_t smem, cudaStream_t stream) {
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

template <bool HOLD>
void (*rows_kernel_of(const VerifyParams& p))(VerifyParams) {
  const bool x = p.target.bf16 != 0, y = p.draft.bf16 != 0;
  if (p.greedy) return x ? rows_kernel<true, true, kGreedy, HOLD> : rows_kernel<false, false, kGreedy, HOLD>;
  if (p.draft.data == nullptr) return x ? rows_kernel<true, true, kLookup, HOLD> : rows_kernel<false, false, kLookup, HOLD>;
  if (x) return y ? rows_kernel<true, true, kDrafted, HOLD> : rows_kernel<true, false, kDrafted, HOLD>;
  return y ? rows_kernel<false, true, kDrafted, HOLD> : rows_kernel<false, false, kDrafted, HOLD>;
}

// Shared memory of a CTA: its part of the target's row in whole groups, and
// the draft's elements of the same places, each warp's with up to 16 bytes on both sides.
int64_t part_bytes(const VerifyParams& p, int ranks) {
  const int64_t groups = (p.vocab + 14) / 8, per = (groups + ranks - 1) / ranks;
  const int64_t x = per * 8 * (p.target.bf16 ? 2 : 4);
  return p.draft.data == nullptr ? x : x + per * 8 * (p.draft.bf16 ? 2 : 4) + 32 * kRowWarps;
}

constexpr int64_t kMostHeld = 220 << 10;   // what a CTA can have, less its static part
constexpr int64_t kGoodPart = 72 << 10;    // three CTAs an SM: one copies while others compute
constexpr int64_t kLeastPart = 8 << 10;

}  // namespace

cudaError_t launch_verify(const VerifyParams& q, cudaStream_t stream) {
  VerifyParams p = q;
  const int64_t rows = p.n_drafts + p.n_seq, sms = device_sms();
  p.ranks = 1;
  while (p.ranks < kMaxRanks && part_bytes(p, p.ranks) > kGoodPart) p.ranks *= 2;
  // few rows: spread over all SMs
  while (p.ranks < kMaxRanks && rows * p.ranks * 2 <= 2 * sms && part_bytes(p, 2 * p.ranks) >= kLeastPart) p.ranks *= 2;
  while (p.ranks > 1 && rows * p.ranks > 0x7fffffff) p.ranks /= 2;
  const int64_t part = part_bytes(p, p.ranks);
  const bool hold = part <= kMostHeld;
  void (*kernel)(VerifyParams) = hold ? rows_kernel_of<true>(p) : rows_kernel_of<false>(p);
  const size_t smem = hold ? size_t(part) : 0;
  if (smem > (40 << 10)) {
    const cudaError_t err = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, int(kMostHeld));
    if (err != cudaSuccess) return err;
  }
  // more rows than run at once: by their place in their sequence, and not behind a draft that fell
  const bool waves = rows * p.ranks > 3 * sms && p.n_drafts > 0;
  p.pitch = waves ? (rows + p.n_seq - 1) / p.n_seq : 1;
  if ((rows + p.pitch) * p.ranks > 0x7fffffff) p.pitch = 1;
  if (!waves) p.fallen = nullptr;
  cudaError_t err = status_ref(&p.status_word, &p.status_host);
  if (err == cudaSuccess && waves) err = launch_after(clear_kernel, p, (p.n_seq + 255) / 256, 256, 1, 0, stream);
  const int64_t items = (rows + p.pitch - 1) / p.pitch * p.pitch;
  if (err == cudaSuccess) err = launch_after(kernel, p, items * p.ranks, kRowThreads, p.ranks, smem, stream);
  if (err == cudaSuccess) err = launch_after(tokens_kernel, p, (p.n_seq + 7) / 8, 256, 1, 0, stream);
  return err;
}

}  // namespace ar
