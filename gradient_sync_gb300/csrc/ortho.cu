// The orthogonalised update: Newton-Schulz steps on tensor cores, and the
// optimiser step around them.
//
// X = U / (|U|_F + eps), then a few times
//   A = X X^T,  B = b A + c A A,  X <- a X + B X
// with m = min(rows, cols) rows (a tall matrix is held transposed). The
// singular values of X go through the odd polynomial a s + b s^3 + c s^5.
//
// Precision. Operands are fp16 with power-of-two scales, accumulators fp32.
// After the normalisation |X| <= 1 and the singular values stay below a bound
// that the plan checks, so fp16's range holds every operand at a fixed scale,
// with 8 times less rounding than bf16. X itself is held as two fp16 numbers
// (hi + lo, 22 bits): a X and the addition of B X are done on those, so that
// the rounding of operands enters through B X only and small singular values,
// which the steps amplify by up to a each, are not drowned. "Split" precision
// also multiplies with both halves: hi hi + hi lo + lo hi, for fp32 results.
// In the last two steps, where most singular values are near 1 and b + c is
// near -2.7, a multiple of the identity moves from a X into B (t in
// OrthoPoly): a X and B X then cancel less and the operands' rounding counts
// half. (Errors of the result against 64 bits, Gaussian 512 x 2048: 1.7e-3
// without, 1.2e-3 with it; fp16 X: 2.9e-3 on a spectrum falling like 1/k.)
//
// Layout. Every operand is stored as blocks of 128 rows x 64 columns (16 KB),
// in the 128-byte-swizzled order that the tensor core reads from shared
// memory, so a tile is one contiguous bulk copy. (Pairs of CTAs copy through a
// tensor map over the same bytes, so that both CTAs' copies count on one barrier.)
// The same bytes serve both ways round: 128 rows of 64 along k (k-major), or
// 64 of the 128 rows as k of 128 columns (two blocks side by side, mn-major).
// X is therefore stored once for X X^T and for B X, and of the symmetric A and
// B only the tiles on and below the diagonal are computed and stored: a tile
// above it is the one below, read the other way round. That leaves
// m^2 n + m^3 + 2 m^2 n operations of a step's 2 m^2 n + 2 m^3 + 2 m^2 n.
//
// Kernels (three launches for all matrices of a call):
//  squares_kernel  momentum update, partial sums of squares of the update. HBM:
//                  111 us for one transformer layer's 67 M elements (fp32
//                  gradients and momentum: 806 MB, 1.07 of the copy bandwidth)
//  pack_kernel     X in blocks, scaled, transposed where tall. HBM: 126 us for
//                  the same (805 MB, 0.94)
//  steps_kernel    every product of every step (ortho_steps.cuh)
#include "ortho_table.cuh"

namespace ar {
namespace {

// ---------------------------------------------------------------- squares

// Sums of squares over all of fp32's range: elements above 2^40 are squared as
// u 2^-85, those below 2^-40 as u 2^85, and the three sums kept apart. With up
// to 2^35 elements none overflows, and what an underflow takes from one is
// nothing beside the element that chose it.
enum Band : int { kLow = 0, kMiddle = 1, kHigh = 2 };
constexpr float kHighFrom = 0x1p40f, kLowTo = 0x1p-40f, kHighScale = 0x1p-85f, kLowScale = 0x1p85f;

struct Squares {
  float low = 0.0f, middle = 0.0f, high = 0.0f;
  // Adds eight elements, or one, by the largest of them; without a branch, so that loads stay ahead.
  template <int N>
  __device__ __forceinline__ void add(const float (&u)[N]) {
    float top = 0.0f;
#pragma unroll
    for (int k = 0; k < N; ++k) top = fmaxf(top, fabsf(u[k]));
    const bool is_high = top > kHighFrom, is_low = top < kLowTo;  // (zeros, and nothing but NaN, are low)
    const float scale = is_high ? kHighScale : is_low ? kLowScale : 1.0f;
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < N; ++k) sum = fmaf(u[k] * scale, u[k] * scale, sum);
    high += is_high ? sum : 0.0f;
    low += is_low ? sum : 0.0f;
    middle += is_high || is_low ? 0.0f : sum;
  }
  __device__ __forceinline__ void add(float value, int band) {
    if (band == kMiddle) middle += value;
    else if (band == kHigh) high += value;
    else low += value;
  }
  // Over the threads of a CTA of 256, in a fixed order; the result in thread 0 (`all`: in all threads).
  __device__ __forceinline__ void reduce(bool all) {
    __shared__ float4 parts[8];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) middle += __shfl_xor_sync(~0u, middle, o);
    if (__any_sync(~0u, low != 0.0f || high != 0.0f)) {  // (not in most calls)
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        low += __shfl_xor_sync(~0u, low, o);
        high += __shfl_xor_sync(~0u, high, o);
      }
    }
    if (threadIdx.x % 32 == 0) parts[threadIdx.x / 32] = make_float4(low, middle, high, 0.0f);
    __syncthreads();
    if (!all && threadIdx.x != 0) return;
    low = middle = high = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      const float4 q = parts[w];
      low += q.x, middle += q.y, high += q.z;
    }
  }
  // The sum as value / scale^2 for the scale of one band; a NaN in any is in the value.
  __device__ __forceinline__ float joined(int& band) const {
    band = high > 0.0f ? kHigh : middle > 0.0f ? kMiddle : kLow;
    if (low + middle + high != low + middle + high) return __int_as_float(0x7fffffff);
    if (band == kHigh) return high + middle * kHighScale * kHighScale;
    if (band == kMiddle) return middle + low / kLowScale / kLowScale;
    return low;
  }
};
__device__ __forceinline__ float scale_of(int band) {
  return band == kHigh ? kHighScale : band == kLow ? kLowScale : 1.0f;
}

// Eight consecutive elements (vec: aligned to 16 bytes), zeros beyond `n`.
template <bool BF16>
__device__ __forceinline__ void load8(const void* base, int64_t e, int n, bool vec, float (&f)[8]) {
  if (vec) {
    if (BF16) {
      const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + e);
      Lane<true, true>::widen(w, f);
    } else {
      const float4 x = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + e);
      const float4 y = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + e + 4);
      f[0] = x.x, f[1] = x.y, f[2] = x.z, f[3] = x.w, f[4] = y.x, f[5] = y.y, f[6] = y.z, f[7] = y.w;
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = k < n ? load_elem<BF16>(base, e + k) : 0.0f;
  }
}

// What gradients are multiplied by; NaN: they are not finite somewhere and count as 0, whatever they hold.
__device__ __forceinline__ float gradient_scale(const OrthoHyper& h) {
  if (h.clip == nullptr) return h.grad_scale;
  return h.clip[3] != 0.0f ? h.clip[1] * h.grad_scale : __int_as_float(0x7fffffff);
}
__device__ __forceinline__ float scaled(float g, float scale) { return scale == scale ? g * scale : 0.0f; }

// One CTA a chunk of kOrthoChunk consecutive elements of one matrix. With
// momentum: M' = mu M + s G, and the update is M' or s G + mu M'.
template <bool BF16>
__global__ void __launch_bounds__(256) squares_kernel(const __grid_constant__ OrthoTable p) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int item = blockIdx.x, i = find_matrix(p, item);
  const OrthoMat& mat = p.mat[i];
  const OrthoIo& io = p.io[i];
  const int64_t cols = mat.turned ? mat.m : mat.n;
  const int64_t total = int64_t(mat.m) * mat.n;
  if (item == 0)  // the products' counters
    for (int k = threadIdx.x; k <= p.n_mat; k += 256) reinterpret_cast<unsigned int*>(p.ws + p.sync_off)[k] = 0;
  const float scale = gradient_scale(p.hyper);
  const int64_t lo = int64_t(item - p.start[0][i]) * kOrthoChunk, hi = lo + kOrthoChunk < total ? lo + kOrthoChunk : total;
  Squares sum;
  if (io.vec_in) {  // eight elements of one row at a time
#pragma unroll 4
    for (int64_t e = lo + threadIdx.x * 8; e < hi; e += 256 * 8) {
      const int64_t r = io.flat ? 0 : e / cols, c = e - r * cols;
      float u[8];
      load8<BF16>(io.g, r * io.g_ld + c, 8, true, u);
      if (p.hyper.muon) {
        float mom[8];
        load8<false>(io.m, r * io.m_ld + c, 8, true, mom);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          u[k] = scaled(u[k], scale);
          mom[k] = fmaf(p.hyper.mu, mom[k], u[k]);
          u[k] = p.hyper.nesterov ? fmaf(p.hyper.mu, mom[k], u[k]) : mom[k];
        }
        float4* to = reinterpret_cast<float4*>(io.m_out + r * io.m_out_ld + c);
        to[0] = make_float4(mom[0], mom[1], mom[2], mom[3]);
        to[1] = make_float4(mom[4], mom[5], mom[6], mom[7]);
      }
      sum.add(u);
    }
  } else {
    for (int64_t e = lo + threadIdx.x; e < hi; e += 256) {
      const int64_t r = io.flat ? 0 : e / cols, c = e - r * cols;
      float u = load_elem<BF16>(io.g, r * io.g_ld + c);
      if (p.hyper.muon) {
        u = scaled(u, scale);
        const float mom = fmaf(p.hyper.mu, io.m[r * io.m_ld + c], u);
        io.m_out[r * io.m_out_ld + c] = mom;
        u = p.hyper.nesterov ? fmaf(p.hyper.mu, mom, u) : mom;
      }
      const float one[1] = {u};
      sum.add(one);
    }
  }
  sum.reduce(false);
  if (threadIdx.x == 0) {
    int band;
    const float value = sum.joined(band);
    reinterpret_cast<float2*>(p.ws + p.part_off)[mat.part + (item - p.start[0][i])] = make_float2(value, float(band));
  }
}

// ---------------------------------------------------------------- pack

// One CTA a block of X: 128 rows x 64 columns, hi and lo. (Four CTAs an SM: with
// the 80 registers it takes when left alone, three, 139 us for a layer and not 126.)
template <bool BF16>
__global__ void __launch_bounds__(256, 4) pack_kernel(const __grid_constant__ OrthoTable p) {
  __shared__ float tile[64][129];  // [column of X][row of X], tall matrices
  grid_dependency_wait();
  grid_dependents_launch();
  const int item = blockIdx.x, i = find_matrix(p, item);
  const OrthoMat& mat = p.mat[i];
  const OrthoIo& io = p.io[i];

  const float by = gradient_scale(p.hyper);
  // eight elements of row r of the caller's matrix, from column c; n of them exist
  auto update = [&](int64_t r, int64_t c, int n, float (&u)[8]) {
    const bool vec = io.vec_in && n >= 8;
    if (!p.hyper.muon) {
      load8<BF16>(io.g, r * io.g_ld + c, n, vec, u);
      return;
    }
    load8<false>(io.m_out, r * io.m_out_ld + c, n, vec, u);
    if (p.hyper.nesterov) {
      float grad[8];
      load8<BF16>(io.g, r * io.g_ld + c, n, vec, grad);
#pragma unroll
      for (int k = 0; k < 8; ++k) u[k] = fmaf(p.hyper.mu, u[k], scaled(grad[k], by));
    }
  };
  const int local = item - p.start[0][i], rb = local / mat.nb, cb = local - rb * mat.nb;
  const int tid = threadIdx.x;
  float v[4][8];
  if (mat.turned) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {  // X(r, c) = U(c, r)
      const int c = q * 16 + tid / 16, r = tid % 16 * 8;
      const int gr = rb * 128 + r, gc = cb * 64 + c;
      update(gc, gr, gc < mat.n ? mat.m - gr : 0, v[q]);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int k = 0; k < 8; ++k) tile[q * 16 + tid / 16][tid % 16 * 8 + k] = v[q][k];
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int r = q * 32 + tid / 8, c = tid % 8 * 8;
      const int gr = rb * 128 + r, gc = cb * 64 + c;
      update(gr, gc, gr < mat.m ? mat.n - gc : 0, v[q]);
    }
  }
  const float2* part = reinterpret_cast<const float2*>(p.ws + p.part_off) + mat.part;
  Squares sum;
  for (int k = tid; k < mat.n_part; k += 256) sum.add(part[k].x, int(part[k].y));
  sum.reduce(true);  // (the tile is written too)
  int band;
  const float norm = sqrtf(sum.joined(band)), first = scale_of(band);  // the norm times `first`, a power of two
  const float scale = mat.sx / (norm + p.eps * first);
  char* hi = p.ws + mat.x + (int64_t(rb) * mat.nb + cb) * kBlockBytes;
  char* lo = hi + mat.x_bytes;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int r = q * 32 + tid / 8, c = tid % 8;
    if (mat.turned) {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[q][k] = tile[c * 8 + k][r];
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) v[q][k] = v[q][k] * first * scale;
    uint4 h, l;
    split_pair(v[q][0], v[q][1], h.x, l.x);
    split_pair(v[q][2], v[q][3], h.y, l.y);
    split_pair(v[q][4], v[q][5], h.z, l.z);
    split_pair(v[q][6], v[q][7], h.w, l.w);
    *reinterpret_cast<uint4*>(hi + chunk_offset(r, c)) = h;
    *reinterpret_cast<uint4*>(lo + chunk_offset(r, c)) = l;
  }
}

// ---------------------------------------------------------------- launches

// The tensor map of the workspace.
cudaError_t encode_map(CUtensorMap* map, char* ws, int64_t bytes) {
  static const auto encode = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<decltype(&cuTensorMapEncodeTiled)>(f);
  }();
  if (encode == nullptr) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {64, cuuint64_t(bytes / 128)}, strides[1] = {128};
  const cuuint32_t box[2] = {64, 64}, step[2] = {1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, ws, dims, strides, box, step,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Matrices order[first, first + n) of the plan.
cudaError_t run(const ar_ortho_plan_t& plan, int first, int n, const OrthoIo* io, const OrthoHyper& hyper, char* ws,
                cudaStream_t stream) {
  OrthoTable p = {};
  p.ws = ws;
  cudaError_t err = status_ref(&p.status.word, &p.status.host);
  if (err == cudaSuccess && plan.cluster > 1) err = encode_map(&p.map, ws, plan.part_off);
  if (err != cudaSuccess) return err;
  p.hyper = hyper;
  p.eps = plan.eps;
  p.part_off = plan.part_off;
  p.sync_off = plan.sync_off;
  p.out16 = plan.out_dtype == AR_BF16;
  p.n_mat = n;
  for (int i = 0; i < n; ++i) {
    p.mat[i] = plan.mats[plan.order[first + i]];
    p.io[i] = io[plan.order[first + i]];
  }
  const bool in16 = plan.in_dtype == AR_BF16;
  fill_starts(p, 0, [](const OrthoMat& m) { return int64_t(m.n_part); });
  err = launch_after(in16 ? squares_kernel<true> : squares_kernel<false>, p, p.total[0], 256, 0, 1, stream);
  fill_starts(p, 0, [](const OrthoMat& m) { return int64_t(m.mb) * m.nb; });
  if (err == cudaSuccess)
    err = launch_after(in16 ? pack_kernel<true> : pack_kernel<false>, p, p.total[0], 256, 0, 1, stream);
  if (err != cudaSuccess) return err;
  p.steps = int(plan.poly.size());
  std::copy(plan.poly.begin(), plan.poly.end(), p.poly);
  if (plan.cluster == 2) return plan.split ? launch_steps<true, 2>(p, stream) : launch_steps<false, 2>(p, stream);
  return plan.split ? launch_steps<true, 1>(p, stream) : launch_steps<false, 1>(p, stream);
}

}  // namespace

cudaError_t launch_ortho(const ar_ortho_plan_t& plan, const OrthoIo* io, const OrthoHyper& hyper, char* ws,
                         cudaStream_t stream) {
  const int n = int(plan.mats.size());
  cudaError_t err = cudaSuccess;
  for (int first = 0; first < n && err == cudaSuccess; first += kGroup)
    err = run(plan, first, std::min(kGroup, n - first), io, hyper, ws, stream);
  return err;
}

}  // namespace ar
