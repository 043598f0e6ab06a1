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
// memory, so a tile is one contiguous bulk copy and no tensor map is needed.
// The same bytes serve both ways round: 128 rows of 64 along k (k-major), or
// 64 of the 128 rows as k of 128 columns (two blocks side by side, mn-major).
// X is therefore stored once for X X^T and for B X, and of the symmetric A and
// B only the tiles on and below the diagonal are computed and stored: a tile
// above it is the one below, read the other way round. That leaves
// m^2 n + m^3 + 2 m^2 n operations of a step's 2 m^2 n + 2 m^3 + 2 m^2 n.
//
// Kernels:
//  squares_kernel  momentum update, partial sums of squares of the update
//  pack_kernel     X in blocks, scaled, transposed where tall
//  gemm_kernel     one of the three products over all matrices of the call:
//                  persistent CTAs; a producer warp, one thread issuing
//                  tcgen05.mma into one half of TMEM, four epilogue warps
//                  emptying the other.
#include "ortho.h"

#include <cuda_fp16.h>

#include <algorithm>

#include "bulk.cuh"
#include "common.cuh"

namespace ar {
namespace {

constexpr uint32_t kWaitPolls = 1u << 22;
constexpr float kScaleA = 4096.0f;  // A and B are held times this
constexpr int kUnit = 16384;        // one operand unit: 128 rows x 64 of k
// Split products are summed over this many steps of 64 along k in the tensor
// core and added up in registers, hi hi apart from the cross terms: the tensor
// core's fp32 sums round towards zero, and every addition to the large sum
// counts. (Error of X against 64 bits, fp32 1024 x 4096: 4.5e-5 with one sum.)
constexpr int kSegment = 4;

enum Op : int { kGram = 0, kSquare = 1, kApply = 2, kApplyLast = 3 };

// ---------------------------------------------------------------- tensor core

__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }

// Shared-memory descriptor of a 128-byte-swizzled operand. k-major: 8-row
// groups 1024 bytes apart. mn-major: 64-column atoms `unit / 2` bytes apart,
// groups of 8 k 1024 bytes apart.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, bool mn) {
  const uint64_t lbo = mn ? uint64_t(kUnit / 2 >> 4) : 1;
  return uint64_t((addr & 0x3FFFF) >> 4) | (lbo << 16) | (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) |
         (uint64_t(2) << 61);
}

// fp16 x fp16 -> fp32, M = 128.
__device__ __forceinline__ uint32_t instr_desc(int n, bool a_mn, bool b_mn) {
  return (1u << 4) | (uint32_t(a_mn) << 15) | (uint32_t(b_mn) << 16) | (uint32_t(n / 8) << 17) | (uint32_t(128 / 16) << 24);
}

__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n"
      ".reg .pred p;\n"
      "setp.ne.u32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n"
      "}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(uint32_t(add))
      : "memory");
}

__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

// 32 consecutive fp32 columns of this warp's 32 accumulator rows, one row a lane.
__device__ __forceinline__ void tmem_load32(uint32_t addr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,"
      "%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// ---------------------------------------------------------------- halves

__device__ __forceinline__ uint32_t half2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ float2 half2_floats(uint32_t w) { return __half22float2(*reinterpret_cast<__half2*>(&w)); }

// v = hi + lo with hi = fp16(v), lo = fp16(v - hi): 22 bits of v.
__device__ __forceinline__ void split_pair(float x, float y, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x, y);
  const float2 f = __half22float2(h);
  hi = half2_bits(h);
  lo = half2_bits(__floats2half2_rn(x - f.x, y - f.y));
}

// Byte offset of 16-byte chunk `c` (0..7) of row `r` in a block.
__device__ __forceinline__ int chunk_offset(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

// ---------------------------------------------------------------- parameters

template <int MAX>
struct OrthoTable {
  char* ws;
  StatusRef status;
  OrthoHyper hyper;
  OrthoPoly poly;
  float eps;
  int64_t part_off;
  int n_mat, total, parity, split;
  OrthoMat mat[MAX];
  OrthoIo io[MAX];
  int32_t start[MAX + 1];  // first work item of each matrix
};

template <class P>
__device__ __forceinline__ int find_matrix(const P& p, int item) {
  int lo = 0, hi = p.n_mat - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (p.start[mid] <= item) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

template <bool BF16>
__device__ __forceinline__ float load_elem(const void* base, int64_t e) {
  if (BF16) return bf16_to_f32(static_cast<const uint16_t*>(base)[e]);
  return static_cast<const float*>(base)[e];
}
template <bool BF16>
__device__ __forceinline__ void store_elem(void* base, int64_t e, float v) {
  if (BF16) static_cast<uint16_t*>(base)[e] = f32_to_bf16(v);
  else static_cast<float*>(base)[e] = v;
}

// ---------------------------------------------------------------- squares

// One CTA a chunk of kOrthoChunk consecutive elements of one matrix. With
// momentum: M' = mu M + s G, and the update is M' or s G + mu M'.
template <int MAX, bool BF16>
__global__ void __launch_bounds__(256) squares_kernel(const __grid_constant__ OrthoTable<MAX> p) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int item = blockIdx.x, i = find_matrix(p, item);
  const OrthoMat& mat = p.mat[i];
  const OrthoIo& io = p.io[i];
  const int64_t cols = mat.turned ? mat.m : mat.n;
  const int64_t total = int64_t(mat.m) * mat.n;
  const int64_t lo = int64_t(item - p.start[i]) * kOrthoChunk, hi = lo + kOrthoChunk < total ? lo + kOrthoChunk : total;
  float sum = 0.0f;
  for (int64_t e = lo + threadIdx.x; e < hi; e += 256) {
    const int64_t r = e / cols, c = e - r * cols;
    float u = load_elem<BF16>(io.g, r * io.g_ld + c);
    if (p.hyper.muon) {
      u *= p.hyper.grad_scale;
      const float mom = fmaf(p.hyper.mu, io.m[r * io.m_ld + c], u);
      io.m_out[r * io.m_out_ld + c] = mom;
      u = p.hyper.nesterov ? fmaf(p.hyper.mu, mom, u) : mom;
    }
    sum = fmaf(u, u, sum);
  }
  __shared__ float parts[8];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
  if (threadIdx.x % 32 == 0) parts[threadIdx.x / 32] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 8; ++w) sum += parts[w];
    reinterpret_cast<float*>(p.ws + p.part_off)[mat.part + (item - p.start[i])] = sum;
  }
}

// ---------------------------------------------------------------- pack

// One CTA a block of X: 128 rows x 64 columns, hi and lo.
template <int MAX, bool BF16>
__global__ void __launch_bounds__(256) pack_kernel(const __grid_constant__ OrthoTable<MAX> p) {
  __shared__ float tile[64][129];  // [column of X][row of X], tall matrices
  __shared__ double parts[8];
  grid_dependency_wait();
  grid_dependents_launch();
  const int item = blockIdx.x, i = find_matrix(p, item);
  const OrthoMat& mat = p.mat[i];
  const OrthoIo& io = p.io[i];
  const float* part = reinterpret_cast<const float*>(p.ws + p.part_off) + mat.part;
  double sum = 0.0;
  for (int k = threadIdx.x; k < mat.n_part; k += 256) sum += double(part[k]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
  if (threadIdx.x % 32 == 0) parts[threadIdx.x / 32] = sum;
  __syncthreads();
  sum = 0.0;
  for (int w = 0; w < 8; ++w) sum += parts[w];
  const float scale = mat.sx / (sqrtf(float(sum)) + p.eps);

  auto update = [&](int64_t r, int64_t c) {  // of the matrix as the caller holds it
    if (!p.hyper.muon) return load_elem<BF16>(io.g, r * io.g_ld + c);
    const float mom = io.m_out[r * io.m_out_ld + c];
    if (!p.hyper.nesterov) return mom;
    return fmaf(p.hyper.mu, mom, load_elem<BF16>(io.g, r * io.g_ld + c) * p.hyper.grad_scale);
  };
  const int local = item - p.start[i], rb = local / mat.nb, cb = local - rb * mat.nb;
  if (mat.turned) {
    for (int e = threadIdx.x; e < 64 * 128; e += 256) {
      const int c = e / 128, r = e % 128;  // X(r, c) = U(c, r)
      const int gr = rb * 128 + r, gc = cb * 64 + c;
      tile[c][r] = gr < mat.m && gc < mat.n ? update(gc, gr) : 0.0f;
    }
    __syncthreads();
  }
  char* hi = p.ws + mat.x + (int64_t(rb) * mat.nb + cb) * kBlockBytes;
  char* lo = hi + mat.x_bytes;
  for (int e = threadIdx.x; e < 128 * 8; e += 256) {
    const int r = e / 8, c = e % 8;
    const int gr = rb * 128 + r, gc = cb * 64 + c * 8;
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (mat.turned) v[k] = tile[c * 8 + k][r];
      else v[k] = gr < mat.m && gc + k < mat.n ? update(gr, gc + k) : 0.0f;
      v[k] *= scale;
    }
    uint4 h, l;
    split_pair(v[0], v[1], h.x, l.x);
    split_pair(v[2], v[3], h.y, l.y);
    split_pair(v[4], v[5], h.z, l.z);
    split_pair(v[6], v[7], h.w, l.w);
    *reinterpret_cast<uint4*>(hi + chunk_offset(r, c)) = h;
    *reinterpret_cast<uint4*>(lo + chunk_offset(r, c)) = l;
  }
}

// ---------------------------------------------------------------- products

// Tiles of one matrix's product: 128 rows x up to NU * 128 columns. The
// symmetric products have those that touch the lower triangle.
template <int OP, int NU>
__host__ __device__ inline int tiles_of(int mb, int nb) {
  if (OP >= kApply) return mb * ((nb / 2 + NU - 1) / NU);
  int n = 0;
  for (int t = 0; t < mb; ++t) n += t / NU + 1;
  return n;
}

struct Tile {
  int i;       // matrix
  int tm, tn;  // first row block; first column block (of 128)
  int nu;      // column blocks
  int steps;   // 64-wide steps along k
};

template <int OP, int NU, class P>
__device__ __forceinline__ Tile find_tile(const P& p, int item) {
  Tile t;
  t.i = find_matrix(p, item);
  const OrthoMat& mat = p.mat[t.i];
  int local = item - p.start[t.i];
  if (OP >= kApply) {
    t.tm = local % mat.mb;
    t.tn = local / mat.mb * NU;
    t.nu = min(NU, mat.nb / 2 - t.tn);
    t.steps = 2 * mat.mb;
  } else {
    t.tm = 0;
    while (local > t.tm / NU) local -= t.tm++ / NU + 1;
    t.tn = local * NU;
    t.nu = min(NU, t.tm - t.tn + 1);
    t.steps = OP == kGram ? mat.nb : 2 * mat.mb;
  }
  return t;
}

// 4 epilogue warps a column block, producer, MMA.
constexpr int gemm_threads(int nu) { return 128 * nu + 64; }

template <int OP, bool SPLIT, int NU, int MAX, bool BF16>
__global__ void __launch_bounds__(gemm_threads(NU), 1) gemm_kernel(const __grid_constant__ OrthoTable<MAX> p) {
  constexpr int HALVES = SPLIT ? 2 : 1;
  constexpr int STAGE = HALVES * (1 + NU) * kUnit;
  constexpr int EPI = 4 * NU;  // epilogue warps
  static_assert(!SPLIT || NU == 1, "the cross terms take the second 128 columns");
  constexpr int SEGMENT = SPLIT ? kSegment : 1 << 30;
  constexpr int STAGES = (224 * 1024 - EPI * 8192) / STAGE;
  extern __shared__ char smem_raw[];
  __shared__ uint64_t full[STAGES], empty[STAGES], acc_full[2], acc_empty[2], done, old_full[EPI];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  volatile int* abort = &abort_flag;
  char* stage0 = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  char* staging = stage0 + STAGES * STAGE;  // 8 KB a warp of the epilogue

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&acc_full[s], 1);
      mbar_init(&acc_empty[s], EPI);
    }
    for (int w = 0; w < EPI; ++w) mbar_init(&old_full[w], 1);
    mbar_init(&done, 1);
    abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == EPI + 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = tmem_slot;
  grid_dependency_wait();
  grid_dependents_launch();
  asm volatile("fence.proxy.async;" ::: "memory");

  if (warp == EPI && lane == 0) {
    // ---- producer
    int it = 0;
    for (int item = blockIdx.x; item < p.total && !*abort; item += gridDim.x) {
      const Tile t = find_tile<OP, NU>(p, item);
      const OrthoMat& mat = p.mat[t.i];
      const char* x = p.ws + mat.x + p.parity * 2 * mat.x_bytes;
      const char* sym = p.ws + mat.a + (OP >= kApply ? HALVES * mat.a_bytes : 0);
      for (int k = 0; k < t.steps; ++k, ++it) {
        const int s = it % STAGES;
        if (it >= STAGES && !mbar_wait(&empty[s], (it / STAGES + 1) & 1, kWaitPolls, abort, p.status)) break;
        mbar_arrive_expect_tx(&full[s], HALVES * (1 + t.nu) * kUnit);
        char* dst = stage0 + s * STAGE;
        // rows `row` x 64 along k: the block itself, or (above the diagonal of
        // a symmetric matrix, or X as the right operand) half a block of each
        // of the two column blocks that hold those rows as columns
        auto load = [&](char* to, const char* base, int nb, int row, bool mn) {
          if (!mn) {
            bulk_load(to, base + (int64_t(row) * nb + k) * kBlockBytes, kUnit, &full[s]);
          } else {
            const char* from = base + (int64_t(k / 2) * nb + 2 * row) * kBlockBytes + (k & 1) * (kUnit / 2);
            bulk_load(to, from, kUnit / 2, &full[s]);
            bulk_load(to + kUnit / 2, from + kBlockBytes, kUnit / 2, &full[s]);
          }
        };
        for (int h = 0; h < HALVES; ++h) {
          const char* a = OP == kGram ? x + h * mat.x_bytes : sym + h * mat.a_bytes;
          load(dst + h * kUnit, a, OP == kGram ? mat.nb : 2 * mat.mb, t.tm, OP != kGram && k / 2 > t.tm);
          const char* b = OP == kSquare ? sym + h * mat.a_bytes : x + h * mat.x_bytes;
          const bool mn = OP >= kApply || (OP == kSquare && k / 2 > t.tn);
          for (int u = 0; u < t.nu; ++u)
            load(dst + (HALVES + h * NU + u) * kUnit, b, OP == kSquare ? 2 * mat.mb : mat.nb, t.tn + u, mn);
        }
      }
    }
    // copies in flight land before the CTA's shared memory goes away
    for (int j = max(0, it - STAGES); j < it; ++j)
      for (uint32_t n = 0; n < kWaitPolls && !mbar_try_wait(&full[j % STAGES], (j / STAGES) & 1); ++n) {
      }
  } else if (warp == EPI + 1 && lane == 0) {
    // ---- tensor core
    int it = 0, part = 0;  // k steps, accumulators filled
    for (int item = blockIdx.x; item < p.total && !*abort; item += gridDim.x) {
      const Tile t = find_tile<OP, NU>(p, item);
      for (int k0 = 0; k0 < t.steps; k0 += SEGMENT, ++part) {
        const int acc = part & 1;
        if (part >= 2 && !mbar_wait(&acc_empty[acc], (part / 2 + 1) & 1, kWaitPolls, abort, p.status)) break;
        fence_after();
        const uint32_t d = tmem + acc * 256;
        for (int k = k0; k < t.steps && k < k0 + SEGMENT; ++k, ++it) {
          const int s = it % STAGES;
          if (!mbar_wait(&full[s], (it / STAGES) & 1, kWaitPolls, abort, p.status)) break;
          fence_after();
          const uint32_t base = smem_u32(stage0 + s * STAGE);
          const bool a_mn = OP != kGram && k / 2 > t.tm, b_mn = OP >= kApply || (OP == kSquare && k / 2 > t.tn);
          const uint32_t idesc = instr_desc(t.nu * 128, a_mn, b_mn);
          const uint64_t a_step = (a_mn ? 2048 : 32) >> 4, b_step = (b_mn ? 2048 : 32) >> 4;
          const uint64_t a0 = operand_desc(base, a_mn), b0 = operand_desc(base + HALVES * kUnit, b_mn);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            mma_f16(d, a0 + j * a_step, b0 + j * b_step, idesc, k > k0 || j > 0);
            if (SPLIT) {
              const uint64_t a1 = operand_desc(base + kUnit, a_mn);
              const uint64_t b1 = operand_desc(base + (HALVES + NU) * kUnit, b_mn);
              mma_f16(d + 128, a0 + j * a_step, b1 + j * b_step, idesc, k > k0 || j > 0);
              mma_f16(d + 128, a1 + j * a_step, b0 + j * b_step, idesc, true);
            }
          }
          mma_commit(&empty[s]);
        }
        mma_commit(&acc_full[acc]);
      }
    }
    // everything issued has finished before TMEM is freed
    mma_commit(&done);
    for (uint32_t n = 0; n < kWaitPolls && !mbar_try_wait(&done, 0); ++n) {
    }
  } else if (warp < EPI) {
    // ---- epilogue
    char* buf = staging + warp * 8192;  // hi, lo of 32 rows x 64 columns
    const int unit = warp / 4, quad = warp % 4;
    uint32_t old_phase = 0;
    int part = 0;
    for (int item = blockIdx.x; item < p.total; item += gridDim.x) {
      const Tile t = find_tile<OP, NU>(p, item);
      const OrthoMat& mat = p.mat[t.i];
      const int row = t.tm * 128 + quad * 32 + lane;
      float sum[SPLIT ? 128 : 1];
      uint32_t at = 0;  // this warp's accumulator
      for (int k0 = 0; k0 < t.steps; k0 += SEGMENT, ++part) {
        const int acc = part & 1;
        const bool ok = mbar_wait(&acc_full[acc], (part / 2) & 1, kWaitPolls, abort, p.status);
        if (__any_sync(~0u, !ok)) goto out;
        fence_after();
        at = tmem + (uint32_t(quad * 32) << 16) + acc * 256 + unit * 128;
        if (SPLIT) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float v[32];
            tmem_load32(at + 128 + q * 32, v);
#pragma unroll
            for (int e = 0; e < 32; ++e) sum[q * 32 + e] = k0 == 0 ? v[e] : sum[q * 32 + e] + v[e];
            tmem_load32(at + q * 32, v);
#pragma unroll
            for (int e = 0; e < 32; ++e) sum[q * 32 + e] += v[e];
          }
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&acc_empty[acc]);
        }
      }
      if (unit >= t.nu) {  // no such column block in this tile
        if (!SPLIT) {
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&acc_empty[(part - 1) & 1]);
        }
        continue;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int cb = 2 * (t.tn + unit) + h;  // block of 64 columns
        char* x_old = p.ws + mat.x + p.parity * 2 * mat.x_bytes;
        char* sym = p.ws + mat.a;
        const int64_t block = (int64_t(t.tm) * (OP >= kApply ? mat.nb : 2 * mat.mb) + cb) * kBlockBytes + quad * 4096;
        // what the result adds to: the tile of A, or of X
        if (OP != kGram) {
          if (lane == 0) {
            bulk_wait_read<0>();
            const bool two = OP >= kApply || SPLIT;
            mbar_arrive_expect_tx(&old_full[warp], two ? 8192 : 4096);
            const char* from = (OP == kSquare ? sym : x_old) + block;
            bulk_load(buf, from, 4096, &old_full[warp]);
            if (two) bulk_load(buf + 4096, from + (OP == kSquare ? mat.a_bytes : mat.x_bytes), 4096, &old_full[warp]);
          }
          const bool landed = mbar_wait(&old_full[warp], old_phase, kWaitPolls, abort, p.status);
          old_phase ^= 1;
          if (__any_sync(~0u, !landed)) {  // winding down: the copy still lands before the CTA goes
            for (uint32_t n = 0; n < kWaitPolls && !mbar_try_wait(&old_full[warp], old_phase ^ 1); ++n) {
            }
            goto out;
          }
        } else if (lane == 0) {
          bulk_wait_read<0>();
        }
        __syncwarp();
        float v[64];
        if (SPLIT) {
#pragma unroll
          for (int e = 0; e < 64; ++e) v[e] = sum[h * 64 + e];
        } else {
          tmem_load32(at + h * 64, *reinterpret_cast<float(*)[32]>(&v[0]));
          tmem_load32(at + h * 64 + 32, *reinterpret_cast<float(*)[32]>(&v[32]));
          if (h == 1) {  // the accumulator is in registers
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[(part - 1) & 1]);
          }
        }
        float scale, add;  // result = scale * accumulator + add * old (in the scale that it is held in)
        if (OP == kGram) {
          scale = kScaleA / (mat.sx * mat.sx);
          add = 0.0f;
        } else if (OP == kSquare) {
          scale = p.poly.c / kScaleA;
          add = p.poly.b;
        } else {
          scale = 1.0f / kScaleA;
          add = p.poly.a - p.poly.t;
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const int off = chunk_offset(lane, c);
          if (OP != kGram) {
            const uint4 hi = *reinterpret_cast<const uint4*>(buf + off);
            uint4 lo = make_uint4(0, 0, 0, 0);
            if (OP >= kApply || SPLIT) lo = *reinterpret_cast<const uint4*>(buf + 4096 + off);
            const uint32_t hw[4] = {hi.x, hi.y, hi.z, hi.w}, lw[4] = {lo.x, lo.y, lo.z, lo.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 a = half2_floats(hw[e]), b = half2_floats(lw[e]);
              v[c * 8 + 2 * e] = fmaf(add, a.x + b.x, v[c * 8 + 2 * e] * scale);
              v[c * 8 + 2 * e + 1] = fmaf(add, a.y + b.y, v[c * 8 + 2 * e + 1] * scale);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[c * 8 + e] *= scale;
          }
        }
        if (OP == kSquare && p.poly.t != 0.0f) {  // + t I
#pragma unroll
          for (int e = 0; e < 64; ++e)
            if (cb * 64 + e == row) v[e] += p.poly.t * kScaleA;
        }
        if (OP != kApplyLast) {
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const int off = chunk_offset(lane, c);
            uint4 hi, lo;
            split_pair(v[c * 8], v[c * 8 + 1], hi.x, lo.x);
            split_pair(v[c * 8 + 2], v[c * 8 + 3], hi.y, lo.y);
            split_pair(v[c * 8 + 4], v[c * 8 + 5], hi.z, lo.z);
            split_pair(v[c * 8 + 6], v[c * 8 + 7], hi.w, lo.w);
            *reinterpret_cast<uint4*>(buf + off) = hi;
            if (OP == kApply || SPLIT) *reinterpret_cast<uint4*>(buf + 4096 + off) = lo;
          }
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) {
            char* to;
            int64_t lo_at;
            if (OP == kApply) {
              to = p.ws + mat.x + (p.parity ^ 1) * 2 * mat.x_bytes + block;
              lo_at = mat.x_bytes;
            } else {
              to = sym + (OP == kSquare ? HALVES * mat.a_bytes : 0) + block;
              lo_at = mat.a_bytes;
            }
            bulk_store(to, buf, 4096);
            if (OP == kApply || SPLIT) bulk_store(to + lo_at, buf + 4096, 4096);
            bulk_commit();
          }
        } else {
          // the result, or the weights' update, in the caller's layout
          const OrthoIo& io = p.io[t.i];
          const float alpha = io.alpha / mat.sx;
          auto put = [&](int64_t r, int64_t c, float value) {
            value *= alpha;
            if (io.w != nullptr) value = fmaf(p.hyper.keep, load_elem<BF16>(io.w, r * io.w_ld + c), value);
            store_elem<BF16>(io.w_out, r * io.w_out_ld + c, value);
          };
          if (mat.turned) {
            // X(row, col) is element (col, row): lanes are consecutive
            if (row < mat.m)
#pragma unroll
              for (int e = 0; e < 64; ++e)
                if (cb * 64 + e < mat.n) put(cb * 64 + e, row, v[e]);
          } else {
            // through shared memory, so that lanes are consecutive columns
            float* words = reinterpret_cast<float*>(buf);
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 64; ++e) words[lane * 64 + (e ^ lane)] = v[e];
            __syncwarp();
            for (int r = 0; r < 32; ++r) {
              const int gr = t.tm * 128 + quad * 32 + r;
              if (gr >= mat.m) break;
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                const int gc = cb * 64 + q * 32 + lane;
                if (gc < mat.n) put(gr, gc, words[r * 64 + ((q * 32 + lane) ^ r)]);
              }
            }
          }
          fence_proxy_async();  // before the next bulk copy into the buffer
          __syncwarp();
        }
      }
    }
  out:
    if (lane == 0) bulk_wait_all();
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if (warp == EPI + 1) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
  }
}

// ---------------------------------------------------------------- launches

template <class P>
cudaError_t launch_after(void (*kernel)(P), const P& p, int grid, int threads, size_t smem, cudaStream_t stream) {
  if (grid <= 0) return cudaSuccess;
  if (smem > 48 * 1024) {
    const cudaError_t err =
        cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel), cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (err != cudaSuccess) return err;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(grid));
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <class P, class F>
void fill_starts(P& p, F&& items) {
  int64_t n = 0;
  for (int i = 0; i < p.n_mat; ++i) {
    p.start[i] = int32_t(n);
    n += items(p.mat[i]);
  }
  p.start[p.n_mat] = int32_t(n);
  p.total = int(n);
}

template <int OP, bool SPLIT, int MAX, bool BF16>
cudaError_t launch_gemm(OrthoTable<MAX>& p, cudaStream_t stream) {
  constexpr int NU = SPLIT ? 1 : 2;
  fill_starts(p, [](const OrthoMat& m) { return tiles_of<OP, NU>(m.mb, m.nb); });
  const size_t smem = 1024 + 224 * 1024;
  return launch_after<OrthoTable<MAX>>(gemm_kernel<OP, SPLIT, NU, MAX, BF16>, p, std::min(p.total, device_sms()),
                                       gemm_threads(NU), smem, stream);
}

template <int MAX, bool SPLIT>
cudaError_t run(const ar_ortho_plan_t& plan, const OrthoIo* io, const OrthoHyper& hyper, char* ws, cudaStream_t stream) {
  OrthoTable<MAX> p = {};
  p.ws = ws;
  cudaError_t err = status_ref(&p.status.word, &p.status.host);
  if (err != cudaSuccess) return err;
  p.hyper = hyper;
  p.eps = plan.eps;
  p.part_off = plan.part_off;
  p.n_mat = int(plan.mats.size());
  for (int i = 0; i < p.n_mat; ++i) {
    p.mat[i] = plan.mats[plan.order[i]];
    p.io[i] = io[plan.order[i]];
  }
  const bool in16 = plan.in_dtype == AR_BF16, out16 = plan.out_dtype == AR_BF16;
  fill_starts(p, [](const OrthoMat& m) { return int64_t(m.n_part); });
  err = launch_after<OrthoTable<MAX>>(in16 ? squares_kernel<MAX, true> : squares_kernel<MAX, false>, p, p.total, 256, 0,
                                      stream);
  fill_starts(p, [](const OrthoMat& m) { return int64_t(m.mb) * m.nb; });
  if (err == cudaSuccess)
    err = launch_after<OrthoTable<MAX>>(in16 ? pack_kernel<MAX, true> : pack_kernel<MAX, false>, p, p.total, 256, 0,
                                        stream);
  const int steps = int(plan.poly.size());
  for (int k = 0; k < steps && err == cudaSuccess; ++k) {
    p.poly = plan.poly[k];
    p.parity = k & 1;
    err = launch_gemm<kGram, SPLIT, MAX, false>(p, stream);
    if (err == cudaSuccess) err = launch_gemm<kSquare, SPLIT, MAX, false>(p, stream);
    if (err != cudaSuccess) break;
    if (k + 1 < steps) err = launch_gemm<kApply, SPLIT, MAX, false>(p, stream);
    else if (out16) err = launch_gemm<kApplyLast, SPLIT, MAX, true>(p, stream);
    else err = launch_gemm<kApplyLast, SPLIT, MAX, false>(p, stream);
  }
  return err;
}

}  // namespace

cudaError_t launch_ortho(const ar_ortho_plan_t& plan, const OrthoIo* io, const OrthoHyper& hyper, char* ws,
                         cudaStream_t stream) {
  // The table travels with every launch: a short one costs less.
  if (plan.mats.size() <= 16)
    return plan.split ? run<16, true>(plan, io, hyper, ws, stream) : run<16, false>(plan, io, hyper, ws, stream);
  return plan.split ? run<AR_MAX_MATRICES, true>(plan, io, hyper, ws, stream)
                    : run<AR_MAX_MATRICES, false>(plan, io, hyper, ws, stream);
}

}  // namespace ar
