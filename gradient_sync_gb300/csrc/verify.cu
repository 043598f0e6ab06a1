// Verification of drafted tokens against the target's probabilities.
//
// For a row of target logits x with maximum m, p_i = w_i / Z with
//   w_i = 2^((x_i - m) k), k = log2(e) / temperature, Z = sum w_i,
// and alike q for the draft's row. The draft t of the row stands while
// u < p_t / q_t. Where it falls, a token is drawn from max(p_i - q_i, 0),
// that is from w_i - v_i (Z / Z') where positive (v, Z' the draft's): the first index whose
// running sum passes u times the total.
//
// A CTA takes a row of the target with its row of the draft, whether or not the
// drafts before it stand: the rows of a sequence run side by side, and each leaves
// what the sequence would need of it (stands or not, the token drawn, both
// log-probabilities). A second kernel, a warp a sequence, finds the first draft
// that falls and writes the tokens. Bound by HBM for many rows: each is read from
// there once, and by further passes from the L2.
//
// A draw has to put u on the right side of borders that may lie anywhere, also
// between tokens of 1e-6 and less. So its weights are to fp32's last place (the
// fast ones of the sums that only decide about drafts are not): the difference x_i - m
// and its product with k are carried with what fp32 leaves of them, the draft's
// weight is subtracted in one fused operation with a two-part factor, and sums
// beyond 8 terms are in 64 bits.
#include "verify.h"

#include <algorithm>

#include "common.cuh"

namespace ar {
namespace {

constexpr int kRowThreads = 512, kRowWarps = kRowThreads / 32;

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A row as groups of 8 elements that start on 16 aligned bytes: element j of
// group g is 8 g + j - lead, and some of the first and last group's are outside.
struct Row {
  const char* p;
  int64_t n, groups;
  int lead;
  bool bf16;
  float k, k_low;
  __device__ Row(const VerifyRows& r, int64_t row, int64_t vocab) {
    p = r.data + row * r.ld * (r.bf16 ? 2 : 4);
    n = vocab;
    bf16 = r.bf16 != 0;
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    lead = bf16 ? int(at / 2 % 8) : int(at / 4 % 4);
    groups = (lead + n + 7) / 8;
    k = r.k;
    k_low = r.k_low;
  }
  __device__ __forceinline__ float at(int64_t i) const {
    return bf16 ? bf16_to_f32(reinterpret_cast<const uint16_t*>(p)[i]) : reinterpret_cast<const float*>(p)[i];
  }
  // Elements i .. i + 7; -inf for those outside the row.
  __device__ __forceinline__ void load(int64_t i, float (&x)[8]) const {
    const char* q = p + i * (bf16 ? 2 : 4);
    if (i >= 0 && i + 8 <= n && reinterpret_cast<uintptr_t>(q) % 16 == 0) {
      if (bf16) {
        const uint4 r = *reinterpret_cast<const uint4*>(q);
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) x[2 * j] = bf16lo(w[j]), x[2 * j + 1] = bf16hi(w[j]);
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float4 r = reinterpret_cast<const float4*>(q)[h];
          x[4 * h] = r.x, x[4 * h + 1] = r.y, x[4 * h + 2] = r.z, x[4 * h + 3] = r.w;
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = i + j >= 0 && i + j < n ? at(i + j) : -INFINITY;
    }
  }
};

// A warp's groups of the row are one behind the other, so that indexes order
// like (warp, round, lane, element).
struct Piece {
  int64_t lo, hi;
  __device__ Piece(int64_t groups, int warp) {
    const int64_t per = (groups + kRowWarps - 1) / kRowWarps;
    lo = min(groups, warp * per);
    hi = min(groups, lo + per);
  }
};

struct Top {
  float x;
  int32_t at;
  bool bad;  // a NaN or +inf somewhere
};
__device__ __forceinline__ Top join(const Top& a, const Top& b) {
  const bool second = b.x > a.x || (b.x == a.x && b.at < a.at);
  return {second ? b.x : a.x, second ? b.at : a.at, a.bad || b.bad};
}

struct Shared {
  Top tops[kRowWarps];
  double sums[kRowWarps];
  double out;
  float2 logs;
  int32_t found;
};

__device__ Top row_top(const Row& r, Shared& sh) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const Piece piece(r.groups, warp);
  Top top = {-INFINITY, INT32_MAX, false};
  float x[8];
#pragma unroll 2
  for (int64_t g = piece.lo + lane; g < piece.hi; g += 32) {
    const int64_t i = 8 * g - r.lead;
    r.load(i, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (x[j] > top.x) top.x = x[j], top.at = int32_t(i) + j;
      top.bad |= !(x[j] <= 3.4028234e38f);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    top = join(top, {__shfl_xor_sync(~0u, top.x, o), __shfl_xor_sync(~0u, top.at, o), __shfl_xor_sync(~0u, int(top.bad), o) != 0});
  __syncthreads();
  if (lane == 0) sh.tops[warp] = top;
  __syncthreads();
  for (int w = 0; w < kRowWarps; ++w) top = join(top, sh.tops[w]);
  return top;
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// The sum over the CTA, for every thread.
__device__ double block_sum(double v, Shared& sh) {
  v = warp_sum(v);
  __syncthreads();
  if (threadIdx.x % 32 == 0) sh.sums[threadIdx.x / 32] = v;
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = 0.0;
    for (int w = 0; w < kRowWarps; ++w) s += sh.sums[w];
    sh.out = s;
  }
  __syncthreads();
  return sh.out;
}

// 2^((x - m) k) to fp32's last place; 0 below 2^-125.
__device__ __forceinline__ float weight(float x, float m, float k, float k_low) {
  const float d = x - m, t = d * k;
  if (!(t >= -125.0f)) return 0.0f;
  const float back = d - x, left = (x - (d - back)) - (m + back);  // d + left = x - m exactly
  const float n = rintf(t);
  const float f = fmaf(left, k, fmaf(d, k_low, fmaf(d, k, -n)));
  return __int_as_float(__float_as_int(exp2_approx(f)) + (int(n) << 23));
}

// Z of a row with maximum m; FAST: with (x - m) k rounded.
template <bool FAST>
__device__ double row_sum(const Row& r, float m, Shared& sh) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const Piece piece(r.groups, warp);
  double sum = 0.0;
  float x[8];
#pragma unroll 2
  for (int64_t g = piece.lo + lane; g < piece.hi; g += 32) {
    r.load(8 * g - r.lead, x);
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) s += FAST ? exp2_approx((x[j] - m) * r.k) : weight(x[j], m, r.k, r.k_low);
    sum += double(s);
  }
  return block_sum(sum, sh);
}

// log S for S >= 1, one thread.
__device__ double log_of(double s) {
  int e;
  const double f = frexp(s, &e);
  const float g = float(f);
  return double(e) * 0.69314718055994531 + double(logf(g)) + (f - double(g)) / f;
}

// What a token is drawn from: w_i, less the draft's weight (a row, or one token).
enum Less : int { kNothing = 0, kRow = 1, kToken = 2 };
struct Draw {
  Row x, y;
  float mx, my;
  float rho, rho_low;  // Z / Z'
  int64_t token;
  int less;
  __device__ __forceinline__ void weights(int64_t i, float (&w)[8]) const {
    float a[8];
    x.load(i, a);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = weight(a[j], mx, x.k, x.k_low);
    if (less == kRow) {
      y.load(i, a);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float v = weight(a[j], my, y.k, y.k_low);
        w[j] = fmaxf(fmaf(-v, rho_low, fmaf(-v, rho, w[j])), 0.0f);
      }
    } else if (less == kToken) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i + j == token) w[j] = 0.0f;
    }
  }
};

// The first index whose running sum passes u times the total; -1 where there is
// no weight.
__device__ int32_t drawn(const Draw& d, float u, Shared& sh) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const Piece piece(d.x.groups, warp);
  double sum = 0.0;
  float w[8];
  for (int64_t g = piece.lo + lane; g < piece.hi; g += 32) {
    d.weights(8 * g - d.x.lead, w);
    sum += double(((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7])));
  }
  const double total = block_sum(sum, sh);
  if (!(total > 0.0)) return -1;
  const double target = double(u) * total;
  // the warp whose piece the border lies in; behind the last border by rounding: the last with any weight
  int where = -1;
  double before = 0.0, upto = 0.0;
  for (int i = 0; i < kRowWarps; ++i) {
    if (sh.sums[i] > 0.0) {
      where = i;
      before = upto;
      upto += sh.sums[i];
      if (upto > target) break;
    }
  }
  if (warp == where) {
    int32_t last = -1, hit = -1;
    for (int64_t g0 = piece.lo; g0 < piece.hi && hit < 0; g0 += 32) {
      const int64_t i = 8 * (g0 + lane) - d.x.lead;
      double chunk = 0.0;
      if (g0 + lane < piece.hi) {
        d.weights(i, w);
        chunk = double(((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7])));
      }
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
              last = int32_t(i) + j;
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
    if (lane == 0) sh.found = hit >= 0 ? hit : last;
  }
  __syncthreads();
  return sh.found;
}

__device__ __forceinline__ int64_t start_of(const VerifyParams& p, int64_t s) {
  if (p.draft_start == nullptr) return s == 0 ? 0 : p.n_drafts;
  return min(max(p.draft_start[s], int64_t(0)), p.n_drafts);
}

template <bool GREEDY>
__global__ void __launch_bounds__(kRowThreads) rows_kernel(const __grid_constant__ VerifyParams p) {
  grid_dependency_wait();
  grid_dependents_launch();
  __shared__ Shared sh;
  const int64_t row = blockIdx.x;
  // the sequence: the last one whose first row is not behind this one
  int64_t s = -1;
  for (int64_t base = 0; base < p.n_seq; base += kRowThreads) {
    const int64_t i = base + threadIdx.x;
    const int n = __syncthreads_count(i < p.n_seq && start_of(p, i) + i <= row);
    s += n;
    if (n < kRowThreads) break;
  }
  if (s < 0) return;
  const int64_t first = start_of(p, s), count = max(start_of(p, s + 1) - first, int64_t(0)), j = row - s - first;
  if (j < 0 || j > count) return;
  const bool behind = j == count;  // the row behind all drafts
  RowResult* result = p.results + row;
  const int64_t token = behind ? -1 : p.drafts[first + j];
  const Row x(p.target, row, p.vocab);
  const Top top = row_top(x, sh);
  const float nan = __int_as_float(0x7fc00000);
  bool ok = !top.bad && top.x > -INFINITY;
  const bool drafted = !GREEDY && !behind && p.draft.data != nullptr;
  const Row y(drafted ? p.draft : p.target, drafted ? first + j : row, p.vocab);
  Top top_y = top;
  if (drafted) {
    top_y = row_top(y, sh);
    ok = ok && !top_y.bad && top_y.x > -INFINITY;
  }
  if (!ok) {
    if (threadIdx.x == 0) *result = {-1, nan, 0.0f, 0, 0};
    return;
  }
  const double z = row_sum<true>(x, top.x, sh);
  if (GREEDY) {
    if (threadIdx.x == 0) {
      const float lp = float(-log_of(z));
      *result = {top.at, lp, lp, int32_t(!behind && token == top.at), 0};
    }
    return;
  }
  const double zy = drafted ? row_sum<true>(y, top_y.x, sh) : 1.0;
  const bool inside = token >= 0 && token < p.vocab;
  // log-probabilities of the draft, and whether it stands
  __shared__ double log_z;
  __shared__ float draft_logp;
  __shared__ int stands;
  if (threadIdx.x == 0) {
    log_z = log_of(z);
    stands = 0;
    const float xt = inside ? x.at(token) : -INFINITY;
    if (xt > -INFINITY) {
      const double lp = (double(xt) - double(top.x)) * p.target.inv_temp - log_z;
      double lq = 0.0;
      if (drafted) lq = (double(y.at(token)) - double(top_y.x)) * p.draft.inv_temp - log_of(zy);
      const float u = fminf(p.uniforms[row], 0.99999994f);  // (a NaN comes out as a number)
      const float ratio = expf(float(lp - lq));
      draft_logp = float(lp);
      stands = p.uniforms[row] == p.uniforms[row] && (u <= 0.0f || u < ratio);
    }
  }
  __syncthreads();
  if (stands) {
    if (threadIdx.x == 0) *result = {-1, 0.0f, draft_logp, 1, 0};
    return;
  }
  Draw d = {x, y, top.x, top_y.x, 0.0f, 0.0f, token, behind ? kNothing : drafted ? kRow : kToken};
  if (drafted) {
    const double rho = row_sum<false>(x, top.x, sh) / row_sum<false>(y, top_y.x, sh);
    d.rho = float(rho);
    d.rho_low = float(rho - double(d.rho));
  }
  const float last = p.uniforms[s + first + count];
  const float u = fminf(fmaxf(last == last ? last : 0.0f, 0.0f), 0.99999994f);
  int32_t found = drawn(d, u, sh);
  if (found < 0) {
    d.less = kNothing;
    found = drawn(d, u, sh);
  }
  if (threadIdx.x == 0)
    *result = {found, float((double(x.at(found)) - double(top.x)) * p.target.inv_temp - log_z), 0.0f, 0, 0};
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
cudaError_t launch_after(void (*kernel)(VerifyParams), const VerifyParams& p, int64_t grid, int threads, cudaStream_t stream) {
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

}  // namespace

cudaError_t launch_verify(const VerifyParams& p, cudaStream_t stream) {
  cudaError_t err = launch_after(p.greedy ? rows_kernel<true> : rows_kernel<false>, p, p.n_drafts + p.n_seq, kRowThreads, stream);
  if (err == cudaSuccess) err = launch_after(tokens_kernel, p, (p.n_seq + 7) / 8, 256, stream);
  return err;
}

}  // namespace ar
