// The Newton-Schulz steps on tensor cores: one kernel for all products of all
// matrices (see ortho.cu for the method and the layout).
#pragma once

#include <mutex>
#include <utility>
#include <vector>

#include "ortho_table.cuh"

namespace ar {
namespace {

constexpr uint32_t kWaitPolls = 1u << 22;
constexpr float kScaleA = 4096.0f;  // A and B are held times this
constexpr int kUnit = 16384;        // one operand unit: 128 rows x 64 of k
// Split products are summed over a few steps of 64 along k in the tensor core
// and added up in registers, hi hi apart from the cross terms: the tensor core's
// fp32 sums round towards zero, and every addition to the large sum counts.
// Relative error of X against 64 bits and time, 1024 x 4096 and 4096 x 4096:
// one sum 4.5e-5; every 4 steps 6.6e-6, 2.9e-6, 398 us, 2.65 ms; every 2 steps
// 3.7e-6, 1.6e-6, 424 us, 2.81 ms; every step 2.2e-6, 1.1e-6, 497 us, 3.36 ms.
// Elementary fp32 operations: 3.9e-6, 4.4e-6, growing with the length, so long
// products are added up every 4 steps. Short ones, where fp32 operations round
// least, are added up every step, but for A = X X^T, which gains nothing by it
// (every 2 steps, every step and fp32 operations: 300 x 3000 3.4e-6, 2.2e-6,
// 1.9e-6, 267 and 274 us; 130 x 4000 3.4e-6, 1.9e-6, 1.9e-6, 267 and 268 us;
// eight of 512 x 2048 354 and 387 us).
constexpr int kLongSums = 64, kShortSums = 8;
__host__ __device__ constexpr int segment_steps(bool split, bool gram, int ks) {
  return !split ? ks : !gram && ks <= kShortSums ? 1 : ks < kLongSums ? 2 : 4;
}

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

// fp16 x fp16 -> fp32, m x n; bits 15 and 16 tell that an operand is mn-major.
__device__ __forceinline__ uint32_t instr_desc(int m, int n) {
  return (1u << 4) | (uint32_t(n / 8) << 17) | (uint32_t(m / 16) << 24);
}

// PAIR: one product of two CTAs' shared memories into both CTAs' TMEM, issued
// by the first CTA of the pair; commits arrive at both.
template <bool PAIR>
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  if (PAIR)
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        "setp.ne.u32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n"
        "}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(uint32_t(add))
        : "memory");
  else
    asm volatile(
        "{\n"
        ".reg .pred p;\n"
        "setp.ne.u32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n"
        "}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(uint32_t(add))
        : "memory");
}

template <bool PAIR>
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  if (PAIR)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(uint16_t(3))
        : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}

// All 512 columns of TMEM (one CTA an SM), by one warp.
template <bool PAIR>
__device__ __forceinline__ void tmem_alloc(uint32_t* slot) {
  if (PAIR) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  } else {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
}
template <bool PAIR>
__device__ __forceinline__ void tmem_free(uint32_t tmem) {
  if (PAIR) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
  else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
}

// One lane of a converged warp, the same one each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n"
      ".reg .pred p;\n"
      "elect.sync _|p, 0xffffffff;\n"
      "selp.u32 %0, 1, 0, p;\n"
      "}\n"
      : "=r"(one));
  return one != 0;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}

// The address of a shared variable in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}

__device__ __forceinline__ void store_remote(int* p, uint32_t rank, int v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr(p, rank)), "r"(v) : "memory");
}

// When this thread's bulk stores (but for the last group, if `newer`) are
// complete: count them, for whoever reads them next.
__device__ __forceinline__ void signal_complete(unsigned int* count, bool newer) {
  if (newer) asm volatile("cp.async.bulk.wait_group 1;" ::: "memory");
  else bulk_wait_all();  // (complete: visible to this thread, hence to whom the count tells)
  asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(count) : "memory");
}

// `bytes` from global memory into this CTA's shared memory, counted on `bar`.
__device__ __forceinline__ void bulk_load_at(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// 64 rows of 128 bytes (8 KB, contiguous) into this CTA's shared memory; `bar`
// is the address, in either CTA of the pair, of the barrier that counts them.
// A bulk copy without a tensor map can signal its own CTA only.
__device__ __forceinline__ void pair_load(uint32_t dst, const CUtensorMap* map, int row, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
      "%3}], [%4];" ::"r"(dst),
      "l"(map), "r"(0), "r"(row), "r"(bar)
      : "memory");
}

// Arrive at the same barrier in CTA `rank` of the cluster; with `publish`, what
// this thread has written there before is visible to who waits for it (which
// takes a fence across the cluster, about a thousand clocks).
template <bool PUBLISH>
__device__ __forceinline__ void mbar_arrive_remote(uint64_t* bar, uint32_t rank) {
  if (PUBLISH)
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr(bar, rank)) : "memory");
  else
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr(bar, rank)) : "memory");
}

// 16 or 32 consecutive fp32 columns of this warp's 32 accumulator rows, one row a lane.
__device__ __forceinline__ void tmem_load16(uint32_t addr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

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

// ---------------------------------------------------------------- products

// The shape of a product's tiles. A worker is one CTA with a tile of 128 rows,
// or a cluster of two with a tile of 256, each with half of the rows of both
// operands in its shared memory. (Clusters of two such pairs, sharing the right
// operand by multicast, measured the same at 144 of the 152 SMs, which is what
// clusters of four leave in use: a pair's copies keep ahead of its products.)
template <bool SPLIT, int CLUSTER>
struct Shape {
  static constexpr bool PAIR = CLUSTER > 1;
  static constexpr int CTAS = CLUSTER;
  static constexpr int HALVES = SPLIT ? 2 : 1;
  // split: the cross terms take as many columns of TMEM again, twice
  static constexpr int COLS = SPLIT ? 128 : 256;
  static constexpr int NU = COLS / 128;
  // epilogue warps, each with 32 rows x BLOCKS * 64 columns (split: sums of 64
  // columns a thread in registers)
  static constexpr int EPI = 8;
  static constexpr int BLOCKS = COLS / 128;
  static constexpr int THREADS = EPI * 32 + 96;
  static constexpr int B_BYTES = COLS / CTAS * 128;  // right operand, one half of it, per CTA and stage
  static constexpr int STAGE = HALVES * (kUnit + B_BYTES);
  static constexpr int SMEM = 224 * 1024;
  static constexpr int STAGES = (SMEM - EPI * 8192) / STAGE;
  static constexpr int PER_TILE = EPI * CLUSTER;  // epilogue warps that report a tile
};

// Tiles of one matrix's product, `nu` column blocks wide. The symmetric
// products have those that touch the lower triangle of 128 * CTAS square blocks.
// Column blocks that row tile `t` of a symmetric product has.
template <class S>
__host__ __device__ inline int lower_blocks(int t) {
  return (t + 1) * S::CTAS;
}
template <class S>
__host__ __device__ inline int tiles_of(int op, int nu, int mb, int nb) {
  const int rows = mb / S::CTAS;
  if (op == kApply) return rows * ((nb / 2 + nu - 1) / nu);
  int n = 0;
  for (int t = 0; t < rows; ++t) n += (lower_blocks<S>(t) + nu - 1) / nu;
  return n;
}

// Whether the input of a step is held as hi + lo. The last two steps amplify
// little: dropping lo there changes the error of a half-precision result by
// less than its own spread (1.1e-3 either way, Gaussian 512 x 2048), and saves
// 8 of the 18 bytes of lo that an element's five steps move.
template <bool SPLIT>
__device__ __forceinline__ bool has_lo(const OrthoTable& p, int step) {
  return SPLIT || step + 2 < p.steps;
}

// One tile of one product.
struct Tile {
  int op, step;  // product (kNone: no more tiles), Newton-Schulz step
  int i;         // matrix
  int tm, tn;    // row, in tiles; first column block of 128
  int nu;        // column blocks
  int ks;        // 64-wide steps along k
  int need;      // tiles of the matrix that must be complete before
};
constexpr int kTileWords = sizeof(Tile) / 4;

// Work items are numbered step by step and product by product, so that what a
// tile needs has lower numbers.
template <class S>
__device__ __forceinline__ Tile find_tile(const OrthoTable& p, int item) {
  Tile t;
  const int per_step = p.total[0] + p.total[1] + p.total[2];
  t.step = item / per_step;
  item -= t.step * per_step;
  t.op = 0;
  while (item >= p.total[t.op]) item -= p.total[t.op++];
  t.i = find_matrix(p, item, t.op);
  const OrthoMat& mat = p.mat[t.i];
  int local = item - p.start[t.op][t.i];
  const int rows = mat.mb / S::CTAS, nu = p.columns[t.op];
  if (t.op == kApply) {
    t.tm = local % rows;
    t.tn = local / rows * nu;
    t.nu = min(nu, mat.nb / 2 - t.tn);
    t.ks = 2 * mat.mb;
  } else {
    t.tm = 0;
    for (;; ++t.tm) {
      const int n = (lower_blocks<S>(t.tm) + nu - 1) / nu;
      if (local < n) break;
      local -= n;
    }
    t.tn = local * nu;
    t.nu = min(nu, lower_blocks<S>(t.tm) - t.tn);
    t.ks = t.op == kGram ? mat.nb : 2 * mat.mb;
  }
  int count[3];
  for (int q = 0; q < 3; ++q) count[q] = p.start[q][t.i + 1] - p.start[q][t.i];
  t.need = t.step * (count[0] + count[1] + count[2]) + (t.op > 0 ? count[0] : 0) + (t.op > 1 ? count[1] : 0);
  return t;
}

// From which step along k on the rows of the left / right operand are read as
// columns: X as the right operand, and what of A or B lies above the diagonal.
template <class S>
__device__ __forceinline__ int left_mn_from(const Tile& t) {
  return t.op == kGram ? t.ks : (t.tm + 1) * 2 * S::CTAS;
}
template <class S>
__device__ __forceinline__ int right_mn_from(const Tile& t) {
  return t.op == kGram ? t.ks : t.op == kApply ? 0 : (t.tn / S::CTAS + 1) * 2 * S::CTAS;
}

// A 32 x 64 block of the result goes to the caller's layout as
//   result = alpha * X (+ keep * weights).
// Tall matrices: X(row, col) is element (col, row), so the lanes' rows are
// consecutive elements; 16 columns from v. Loads go ahead of the stores, since
// the two may be the same memory.
template <bool BF16>
__device__ __forceinline__ void write_turned(const OrthoIo& io, const OrthoMat& mat, float keep, int row, int col0,
                                             const float (&v)[16]) {
  if (row >= mat.m) return;
  const float alpha = io.alpha / mat.sx;
  float w[16];
#pragma unroll
  for (int e = 0; e < 16; ++e)
    w[e] = io.w != nullptr && col0 + e < mat.n ? load_elem<BF16>(io.w, int64_t(col0 + e) * io.w_ld + row) : 0.0f;
#pragma unroll
  for (int e = 0; e < 16; ++e)
    if (col0 + e < mat.n)
      store_elem<BF16>(io.w_out, int64_t(col0 + e) * io.w_out_ld + row, fmaf(keep, w[e], alpha * v[e]));
}

// Others: from shared memory, where every 8 columns of a row take the 16 + 16
// bytes that their old values had, with lanes along the columns.
template <bool BF16>
__device__ __forceinline__ void write_rows(const OrthoIo& io, const OrthoMat& mat, float keep, int row0, int col0,
                                           const char* buf) {
  constexpr int E = BF16 ? 8 : 4;  // elements of a 16-byte access
  constexpr int LANES = 64 / E, ROWS = 32 / LANES, STEPS = 32 / ROWS, BATCH = 8;  // lanes a row, rows an access
  const int lane = threadIdx.x % 32;
  const float alpha = io.alpha / mat.sx;
  const bool add = io.w != nullptr;
  auto four = [&](int r, int c) {  // columns c .. c + 3 of row r, c a multiple of 4
    return *reinterpret_cast<const float4*>(buf + (c & 4) * 1024 + chunk_offset(r, c / 8));
  };
  if (io.vec_out && col0 + 64 <= mat.n) {
    const int c = lane % LANES * E;
#pragma unroll 1
    for (int s0 = 0; s0 < STEPS; s0 += BATCH) {
      uint4 w[BATCH];
#pragma unroll
      for (int s = 0; s < BATCH; ++s) {
        const int r = (s0 + s) * ROWS + lane / LANES;
        w[s] = make_uint4(0, 0, 0, 0);
        if (add && row0 + r < mat.m)
          w[s] = *reinterpret_cast<const uint4*>(static_cast<const char*>(io.w) +
                                                 (int64_t(row0 + r) * io.w_ld + col0 + c) * (BF16 ? 2 : 4));
      }
#pragma unroll
      for (int s = 0; s < BATCH; ++s) {
        const int r = (s0 + s) * ROWS + lane / LANES;
        float f[E];
        Lane<BF16, true>::widen(w[s], f);
#pragma unroll
        for (int q = 0; q < E; q += 4) {
          const float4 x = four(r, c + q);
          f[q] = fmaf(keep, f[q], alpha * x.x);
          f[q + 1] = fmaf(keep, f[q + 1], alpha * x.y);
          f[q + 2] = fmaf(keep, f[q + 2], alpha * x.z);
          f[q + 3] = fmaf(keep, f[q + 3], alpha * x.w);
        }
        if (row0 + r < mat.m)
          *reinterpret_cast<uint4*>(static_cast<char*>(io.w_out) +
                                    (int64_t(row0 + r) * io.w_out_ld + col0 + c) * (BF16 ? 2 : 4)) =
              Lane<BF16, true>::narrow(f);
      }
    }
    return;
  }
#pragma unroll 1
  for (int r0 = 0; r0 < 32; r0 += 8) {
    float w[8][2];
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int gr = row0 + r0 + r, gc = col0 + q * 32 + lane;
        w[r][q] = add && gr < mat.m && gc < mat.n ? load_elem<BF16>(io.w, int64_t(gr) * io.w_ld + gc) : 0.0f;
      }
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int rr = r0 + r, gr = row0 + rr, c = q * 32 + lane, gc = col0 + c;
        const float x = *reinterpret_cast<const float*>(buf + (c & 4) * 1024 + chunk_offset(rr, c / 8) + c % 4 * 4);
        if (gr < mat.m && gc < mat.n)
          store_elem<BF16>(io.w_out, int64_t(gr) * io.w_out_ld + gc, fmaf(keep, w[r][q], alpha * x));
      }
  }
}

// 16 columns of a row of a tile's result, from the accumulator's values in v:
//   result = scale * accumulator + add * old (+ t I), in the scale that it is held in.
// The old values' place in the buffer (chunks 2 q and 2 q + 1 of the row) takes
// the new ones: as hi and lo, or (last) as fp32.
struct Combine {
  float scale, add, diag;
  bool lo_in, lo_out;  // hi + lo, or hi alone
};
template <int OP, bool SPLIT>
__device__ __forceinline__ Combine combine_of(const OrthoTable& p, const OrthoMat& mat, int step) {
  const OrthoPoly& poly = p.poly[step];
  if (OP == kGram) return {kScaleA / (mat.sx * mat.sx), 0.0f, 0.0f, false, SPLIT};
  if (OP == kSquare) return {poly.c / kScaleA, poly.b, poly.t * kScaleA, SPLIT, SPLIT};
  return {1.0f / kScaleA, poly.a - poly.t, 0.0f, has_lo<SPLIT>(p, step), has_lo<SPLIT>(p, step + 1)};
}
template <int OP, bool SPLIT>
__device__ __forceinline__ void combine16(const Combine& f, int q, int diag, float (&v)[16], char* buf) {
  const int lane = threadIdx.x % 32;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int off = chunk_offset(lane, 2 * q + c);
    float* u = v + 8 * c;
    if (OP != kGram) {
      const uint4 hi = *reinterpret_cast<const uint4*>(buf + off);
      uint4 lo = make_uint4(0, 0, 0, 0);
      if (f.lo_in) lo = *reinterpret_cast<const uint4*>(buf + 4096 + off);
      const uint32_t hw[4] = {hi.x, hi.y, hi.z, hi.w}, lw[4] = {lo.x, lo.y, lo.z, lo.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 a = half2_floats(hw[e]), b = half2_floats(lw[e]);
        u[2 * e] = fmaf(f.add, a.x + b.x, u[2 * e] * f.scale);
        u[2 * e + 1] = fmaf(f.add, a.y + b.y, u[2 * e + 1] * f.scale);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] *= f.scale;
    }
    if (OP == kSquare) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (diag == 16 * q + 8 * c + e) u[e] += f.diag;
    }
    if (OP == kApplyLast) {
      *reinterpret_cast<float4*>(buf + off) = make_float4(u[0], u[1], u[2], u[3]);
      *reinterpret_cast<float4*>(buf + 4096 + off) = make_float4(u[4], u[5], u[6], u[7]);
    } else {
      uint4 hi, lo;
      split_pair(u[0], u[1], hi.x, lo.x);
      split_pair(u[2], u[3], hi.y, lo.y);
      split_pair(u[4], u[5], hi.z, lo.z);
      split_pair(u[6], u[7], hi.w, lo.w);
      *reinterpret_cast<uint4*>(buf + off) = hi;
      if (f.lo_out) *reinterpret_cast<uint4*>(buf + 4096 + off) = lo;
    }
  }
}

// A block of 32 rows x 64 columns: accumulator in TMEM at `at`, or (split) in sum.
template <int OP, bool SPLIT>
__device__ __forceinline__ void finish_block(const OrthoTable& p, const Tile& t, int cb, int row0, int64_t block,
                                             uint32_t at, const float* sum, char* buf) {
  constexpr int HALVES = SPLIT ? 2 : 1;
  const int lane = threadIdx.x % 32;
  const OrthoMat& mat = p.mat[t.i];
  const Combine f = combine_of<OP, SPLIT>(p, mat, t.step);
  const int diag = row0 + lane - cb * 64;
  auto group = [&](int q, float(&v)[16]) {
    combine16<OP, SPLIT>(f, q, diag, v, buf);
    if (OP == kApplyLast && mat.turned) {
      if (p.out16) write_turned<true>(p.io[t.i], mat, p.hyper.keep, row0 + lane, cb * 64 + 16 * q, v);
      else write_turned<false>(p.io[t.i], mat, p.hyper.keep, row0 + lane, cb * 64 + 16 * q, v);
    }
  };
  if (SPLIT) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float v[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] = sum[16 * q + e];
      group(q, v);
    }
  } else {
#pragma unroll 2
    for (int q = 0; q < 4; ++q) {
      float v[16];
      tmem_load16(at + 16 * q, v);
      group(q, v);
    }
  }
  if constexpr (OP == kApplyLast) {
    __syncwarp();
    if (!mat.turned) {
      if (p.out16) write_rows<true>(p.io[t.i], mat, p.hyper.keep, row0, cb * 64, buf);
      else write_rows<false>(p.io[t.i], mat, p.hyper.keep, row0, cb * 64, buf);
    }
    fence_proxy_async();  // before the next bulk copy into the buffer
    __syncwarp();
  } else {
    fence_proxy_async();
    __syncwarp();
    if (lane == 0) {
      char* to;
      int64_t lo_at;
      if (OP == kApply) {
        to = p.ws + mat.x + ((t.step & 1) ^ 1) * 2 * mat.x_bytes + block;
        lo_at = mat.x_bytes;
      } else {
        to = p.ws + mat.a + (OP == kSquare ? HALVES * mat.a_bytes : 0) + block;
        lo_at = mat.a_bytes;
      }
      bulk_store(to, buf, 4096);
      if (f.lo_out) bulk_store(to + lo_at, buf + 4096, 4096);
      bulk_commit();
    }
  }
}

// Waits until `need` of the matrix's tiles are complete. (Copies of what they
// wrote need a proxy fence of the thread that issues them.)
__device__ __forceinline__ bool tiles_complete(const unsigned int* done, unsigned int need, volatile int* abort,
                                               const StatusRef& status) {
  bool ok = false;
  for (uint32_t n = 0; n < kWaitPolls && !*abort; ++n) {
    unsigned int v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(done) : "memory");
    if (v >= need) {
      ok = true;
      break;
    }
    __nanosleep(32);
  }
  if (!ok && !*abort) report_timeout(abort, status);
  return ok;
}

// All steps of all matrices. Workers (CTAs or pairs) take tiles from a queue
// in order. A tile waits for its matrix's earlier products only, and those are
// taken before it, so some worker can always go on, however many run at once;
// and one matrix's tiles fill the others' waits. Of a CTA, one warp takes tiles
// up to two ahead, tells the others of each and, once what it needs is there,
// that it can start; one copies operands; one issues products into one half of
// TMEM; eight empty the other half.
//
// What bounds it, and what it measured (products counted with the symmetric
// ones at one triangle; a 256 x 256 x 64 step of a pair takes 480 clocks, the
// tensor core's rate, when its operands are there):
//  one transformer layer, half precision (4 x 2048 x 2048, 3 x 2048 x 8192):
//  1.8 ms, 1.3 PFLOP/s, 0.69 of the bf16 matrix rate. A tile of the last
//  product of a step takes 20 thousand clocks instead of 16: with its old and
//  new values a CTA moves 78 bytes a clock, and an SM gets about 70 from the
//  L2; 2.5 thousand pass between tiles.
//  two 4096 x 4096: 1.57 PFLOP/s (0.82). 12288 x 4096, split: 7.2 ms, three
//  times the products at 1.43 PFLOP/s (0.75); operands (62 bytes a clock and
//  SM) and the last, partly filled round of each product's tiles.
//  256 x 256: 95 us: 15 products that wait for one another, 12 thousand clocks
//  each: a copy's latency, the epilogue, and the way of a count through the L2.
template <bool SPLIT, int CLUSTER>
__global__ void __launch_bounds__(Shape<SPLIT, CLUSTER>::THREADS, 1)
    steps_kernel(const __grid_constant__ OrthoTable p) {
  using S = Shape<SPLIT, CLUSTER>;
  constexpr bool PAIR = S::PAIR;
  constexpr int HALVES = S::HALVES, EPI = S::EPI, STAGES = S::STAGES, RING = 3;
  extern __shared__ char smem_raw[];
  __shared__ uint64_t full[STAGES], empty[STAGES], acc_full[2], acc_empty[2], done, old_full[EPI];
  __shared__ uint64_t item_full[RING], item_free[RING], item_ready[RING], mail_full[RING], mail_free[RING], mail_ready[RING];
  __shared__ int items[RING][kTileWords], mail[RING][kTileWords];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  volatile int* abort = &abort_flag;
  char* stage0 = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  char* staging = stage0 + STAGES * S::STAGE;  // 8 KB a warp of the epilogue
  unsigned int* queue = reinterpret_cast<unsigned int*>(p.ws + p.sync_off);
  unsigned int* complete = queue + 1;  // per matrix: epilogue warps that have finished a tile

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rank = PAIR ? int(cluster_rank()) : 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&acc_full[s], 1);
      mbar_init(&acc_empty[s], EPI * S::CTAS);
    }
    for (int s = 0; s < RING; ++s) {
      mbar_init(&item_full[s], 1);
      mbar_init(&item_free[s], rank == 0 ? EPI + 2 : EPI + 1);  // epilogue, producer, tensor core
      mbar_init(&item_ready[s], 1);
      mbar_init(&mail_ready[s], 1);
      mbar_init(&mail_full[s], 1);
      mbar_init(&mail_free[s], 1);
    }
    for (int w = 0; w < EPI; ++w) mbar_init(&old_full[w], 1);
    mbar_init(&done, 1);
    abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == EPI + 1) tmem_alloc<PAIR>(&tmem_slot);
  fence_before();
  __syncthreads();
  if (PAIR) cluster_sync();  // the other CTA's barriers exist
  fence_after();
  const uint32_t tmem = tmem_slot;
  grid_dependency_wait();
  grid_dependents_launch();
  asm volatile("fence.proxy.async;" ::: "memory");

  // The n-th tile of this worker, and whether what it needs is there.
  auto receive = [&](int n, Tile& t) {
    const bool ok = mbar_wait(&item_full[n % RING], (n / RING) & 1, kWaitPolls, abort, p.status);
    const volatile int* w = items[n % RING];
    t.op = w[0], t.step = w[1], t.i = w[2], t.tm = w[3], t.tn = w[4], t.nu = w[5], t.ks = w[6];
    return !__any_sync(~0u, !ok) && t.op != kNone;
  };
  auto ready = [&](int n) {
    return !__any_sync(~0u, !mbar_wait(&item_ready[n % RING], (n / RING) & 1, kWaitPolls, abort, p.status));
  };
  auto taken = [&](int n) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&item_free[n % RING]);
  };

  if (warp == EPI + 2) {
    // ---- tiles for the worker: the first CTA takes them and passes them on;
    // each CTA's warps then hear of them from their own CTA only
    if (lane == 0) {
      const int n_items = p.steps * (p.total[0] + p.total[1] + p.total[2]);
      for (int n = 0; !*abort; ++n) {
        const int s = n % RING;
        const uint32_t reuse = (n / RING + 1) & 1;
        int words[7];
        Tile t = {kNone, 0, 0, 0, 0, 0, 0, 0};
        if (rank == 0) {
          const int item = int(atomicAdd(queue, 1u));
          if (item < n_items) t = find_tile<S>(p, item);
          words[0] = t.op, words[1] = t.step, words[2] = t.i, words[3] = t.tm, words[4] = t.tn, words[5] = t.nu;
          words[6] = t.ks;
          if (PAIR) {
            if (n >= RING && !mbar_wait<true>(&mail_free[s], reuse, kWaitPolls, abort, p.status)) break;
#pragma unroll
            for (int w = 0; w < 7; ++w) store_remote(&mail[s][w], 1, words[w]);
            mbar_arrive_remote<true>(&mail_full[s], 1);
          }
        } else {
          if (!mbar_wait<true>(&mail_full[s], (n / RING) & 1, kWaitPolls, abort, p.status)) break;
#pragma unroll
          for (int w = 0; w < 7; ++w) words[w] = *static_cast<volatile int*>(&mail[s][w]);
        }
        if (n >= RING && !mbar_wait(&item_free[s], reuse, kWaitPolls, abort, p.status)) break;
#pragma unroll
        for (int w = 0; w < 7; ++w) items[s][w] = words[w];
        mbar_arrive(&item_full[s]);
        if (words[0] == kNone) break;
        if (rank == 0) {
          if (t.need > 0 && !tiles_complete(complete + t.i, unsigned(t.need) * S::PER_TILE, abort, p.status)) break;
          if (PAIR) mbar_arrive_remote<true>(&mail_ready[s], 1);
        } else {
          if (!mbar_wait<true>(&mail_ready[s], (n / RING) & 1, kWaitPolls, abort, p.status)) break;
          mbar_arrive_remote<true>(&mail_free[s], 0);
        }
        mbar_arrive(&item_ready[s]);
      }
    }
  } else if (warp == EPI) {
    // ---- producer: this CTA's rows of both operands. A step is a handful of
    // copies of 8 KB, one a lane: issued by one thread, one after the other,
    // they took longer (about 150 clocks each) than the products they feed.
    const uint32_t bar0 = PAIR ? cluster_addr(&full[0], 0) : smem_u32(&full[0]);
    int s = 0, steps_issued = 0;
    uint32_t phase = 1;  // the empty barriers' parity: the first round waits for nothing
    // One lane's copies of a tile: half of an operand unit's 128 rows x 64 of k,
    // or (mn) half a block of one of the two column blocks that hold those rows
    // as columns. Places in the workspace count in rows of 128 bytes.
    struct Copies {
      int ks, at_k, at_mn, mn_from, nb;
      uint32_t dst, bytes;
      bool active, whole;  // whole: a k-major unit in one copy of this lane
    };
    auto set_up = [&](const Tile& t, Copies& q) {
      const OrthoMat& mat = p.mat[t.i];
      const bool is_a = lane < 2 * HALVES;
      const int per_half = PAIR ? t.nu : 2 * t.nu;  // copies of the right operand
      const int c = is_a ? lane : lane - 2 * HALVES;
      const int h = is_a ? c / 2 : c / per_half;
      q.active = is_a || h < HALVES;
      int row, sub;  // block of rows, half of it
      if (is_a) {
        row = t.tm * S::CTAS + rank;
        sub = c & 1;
      } else if (!PAIR) {
        row = t.tn + c % per_half / 2;
        sub = c & 1;
      } else if (t.nu == 1) {  // 64 rows a CTA
        row = t.tn;
        sub = rank;
      } else {
        row = t.tn + rank;
        sub = c % per_half;
      }
      q.whole = sub == 0;
      q.dst = smem_u32(stage0) + (is_a ? h * kUnit + sub * (kUnit / 2)
                                       : HALVES * kUnit + h * S::B_BYTES + c % per_half * (kUnit / 2));
      const bool is_x = is_a ? t.op == kGram : t.op != kSquare;
      q.nb = is_x ? mat.nb : 2 * mat.mb;
      const int64_t base = is_x ? mat.x + (t.step & 1) * 2 * mat.x_bytes + h * mat.x_bytes
                                : mat.a + (t.op == kApply ? HALVES * mat.a_bytes : 0) + h * mat.a_bytes;
      q.at_k = int(base / 128) + row * q.nb * 128 + sub * 64;
      q.at_mn = int(base / 128) + row * 256 + sub * 128;
      q.mn_from = is_a ? left_mn_from<S>(t) : right_mn_from<S>(t);
      q.bytes = HALVES * (S::CTAS * kUnit + t.nu * kUnit);
      q.ks = t.ks;
    };
    Tile t;
    Copies q, after;
    bool more = receive(0, t);
    if (more) set_up(t, q);
    for (int n = 0; more; ++n, q = after) {
      if (!ready(n)) break;
      taken(n);
      asm volatile("fence.proxy.async;" ::: "memory");
      // the next tile is prepared while this one's copies wait for room
      const int prepare = min(STAGES, q.ks) - 1;
      for (int k = 0; k < q.ks; ++k) {
        if (!mbar_wait(&empty[s], phase, kWaitPolls, abort, p.status)) break;
        // the second CTA's copies count on the first one's barrier
        if (lane == 0 && rank == 0) mbar_arrive_expect_tx(&full[s], q.bytes);
        const int from = k >= q.mn_from ? q.at_mn + (k >> 1) * q.nb * 128 + (k & 1) * 64 : q.at_k + k * 128;
        const uint32_t to = q.dst + s * S::STAGE, bar = bar0 + s * 8;
        if (q.active) {
          if (PAIR) pair_load(to, &p.map, from, bar);
          else if (k >= q.mn_from) bulk_load_at(to, p.ws + int64_t(from) * 128, kUnit / 2, bar);
          else if (q.whole) bulk_load_at(to, p.ws + int64_t(from) * 128, kUnit, bar);
        }
        ++steps_issued;
        if (++s == STAGES) {
          s = 0;
          phase ^= 1;
        }
        if (k == prepare) {
          __syncwarp();
          more = receive(n + 1, t);
          if (more) set_up(t, after);
        }
      }
      __syncwarp();
    }
    // copies in flight land before the shared memory goes away
    if (lane == 0 && rank == 0)
      for (int j = max(0, steps_issued - STAGES); j < steps_issued; ++j)
        for (uint32_t n = 0; n < kWaitPolls && !mbar_try_wait(&full[j % STAGES], (j / STAGES) & 1); ++n) {
        }
  } else if (warp == EPI + 1 && rank == 0) {
    // ---- tensor core. The whole warp runs the loop, so that descriptors stay
    // in uniform registers, and one elected lane issues: with a branch to a
    // single thread each product took about 90 clocks to issue, more than a
    // 256 x 128 x 16 product takes.
    const bool issue = elect_one();
    int s = 0, part = 0;  // stage, accumulators filled
    uint32_t phase = 0;
    const uint32_t stage_addr = smem_u32(stage0);
    Tile t;
    for (int n = 0; receive(n, t); ++n) {
      taken(n);
      const int a_from = left_mn_from<S>(t), b_from = right_mn_from<S>(t);
      const uint32_t idesc = instr_desc(S::CTAS * 128, t.nu * 128);
      const int segment = segment_steps(SPLIT, t.op == kGram, t.ks);
      for (int k0 = 0; k0 < t.ks; k0 += segment, ++part) {
        const int acc = part & 1;
        if (part >= 2 && __any_sync(~0u, !mbar_wait(&acc_empty[acc], (part / 2 + 1) & 1, kWaitPolls, abort, p.status)))
          break;
        fence_after();
        const uint32_t d = tmem + acc * 256;
        const int k1 = min(t.ks, k0 + segment);
        for (int k = k0; k < k1; ++k) {
          if (__any_sync(~0u, !mbar_wait(&full[s], phase, kWaitPolls, abort, p.status))) break;
          fence_after();
          const bool a_mn = k >= a_from, b_mn = k >= b_from;
          const uint32_t id = idesc | (uint32_t(a_mn) << 15) | (uint32_t(b_mn) << 16);
          const uint32_t a_step = (a_mn ? 2048 : 32) >> 4, b_step = (b_mn ? 2048 : 32) >> 4;
          const uint32_t base = stage_addr + s * S::STAGE;
          const uint64_t a0 = operand_desc(base, a_mn), b0 = operand_desc(base + HALVES * kUnit, b_mn);
          if (issue) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              mma_f16<PAIR>(d, a0 + j * a_step, b0 + j * b_step, id, k > k0 || j > 0);
              if (SPLIT) {
                const uint64_t a1 = a0 + (kUnit >> 4), b1 = b0 + (S::B_BYTES >> 4);
                mma_f16<PAIR>(d + 128, a0 + j * a_step, b1 + j * b_step, id, k > k0 || j > 0);
                mma_f16<PAIR>(d + 128, a1 + j * a_step, b0 + j * b_step, id, true);
              }
            }
            mma_commit<PAIR>(&empty[s]);
            if (k + 1 == k1) mma_commit<PAIR>(&acc_full[acc]);
          }
          __syncwarp();
          if (++s == STAGES) {
            s = 0;
            phase ^= 1;
          }
        }
      }
    }
    // everything issued has finished before TMEM is freed
    if (issue) mma_commit<PAIR>(&done);
    __syncwarp();
    for (uint32_t n = 0; n < kWaitPolls && !mbar_try_wait(&done, 0); ++n) {
    }
  } else if (PAIR && warp == EPI + 1) {
    // ---- the second CTA's products are issued by the first one
    for (uint32_t n = 0; n < kWaitPolls && !mbar_try_wait(&done, 0); ++n) {
    }
  } else if (warp < EPI) {
    // ---- epilogue
    char* buf = staging + warp * 8192;  // hi, lo of 32 rows x 64 columns
    const int part_of = warp / 4, quad = warp % 4;  // columns, rows of the tile
    uint32_t old_phase = 0;
    int part = 0, owed = -1;  // accumulators emptied; matrix of a tile whose completion is still to be told
    auto release = [&](int acc) {  // the accumulator is in registers
      fence_before();
      __syncwarp();
      if (lane == 0) {
        if (PAIR) mbar_arrive_remote<false>(&acc_empty[acc], 0);
        else mbar_arrive(&acc_empty[acc]);
      }
    };
    // The last tile's stores take a while to complete; while more work is at
    // hand it comes first, and the report goes out with the next one's.
    auto report = [&](bool newer) {
      if (owed >= 0 && lane == 0) signal_complete(complete + owed, newer);
      owed = -1;
    };
    auto load_old = [&](const Tile& t, int64_t block) {  // what the result adds to: the tile of A, or of X
      if (lane != 0) return;
      const OrthoMat& mat = p.mat[t.i];
      bulk_wait_read<0>();
      if (t.op == kGram) return;
      const bool two = SPLIT || (t.op == kApply && has_lo<SPLIT>(p, t.step));
      mbar_arrive_expect_tx(&old_full[warp], two ? 8192 : 4096);
      const char* from = p.ws + block + (t.op == kSquare ? mat.a : mat.x + (t.step & 1) * 2 * mat.x_bytes);
      bulk_load(buf, from, 4096, &old_full[warp]);
      if (two) bulk_load(buf + 4096, from + (t.op == kSquare ? mat.a_bytes : mat.x_bytes), 4096, &old_full[warp]);
    };
    Tile t;
    for (int n = 0;; ++n) {
      if (!mbar_test(&item_full[n % RING], (n / RING) & 1)) report(false);
      __syncwarp();
      if (!receive(n, t)) break;
      const OrthoMat& mat = p.mat[t.i];
      const int rb = t.tm * S::CTAS + rank, row0 = rb * 128 + quad * 32;
      // Blocks of 64 columns of this warp: two, or one of a tile of 128 columns.
      const int blocks = min(S::BLOCKS, t.nu);
      const int cb0 = 2 * t.tn + part_of * blocks;
      const int64_t block0 = (int64_t(rb) * (t.op == kApply ? mat.nb : 2 * mat.mb) + cb0) * kBlockBytes + quad * 4096;
      bool landed = true;
      if (!mbar_test(&item_ready[n % RING], (n / RING) & 1)) report(false);
      if (!ready(n)) break;
      taken(n);
      if (lane == 0) asm volatile("fence.proxy.async;" ::: "memory");
      load_old(t, block0);
      float sum[SPLIT ? 64 : 1];
      uint32_t at = 0;  // this warp's accumulator
      const int segment = segment_steps(SPLIT, t.op == kGram, t.ks);
      for (int k0 = 0; k0 < t.ks; k0 += segment, ++part) {
        const int acc = part & 1;
        if (owed >= 0 && !mbar_test(&acc_full[acc], (part / 2) & 1)) report(false);
        __syncwarp();
        const bool ok = mbar_wait(&acc_full[acc], (part / 2) & 1, kWaitPolls, abort, p.status);
        if (__any_sync(~0u, !ok)) {
          landed = false;
          break;
        }
        fence_after();
        at = tmem + (uint32_t(quad * 32) << 16) + acc * 256 + part_of * blocks * 64;
        if (SPLIT) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            float v[32];
            tmem_load32(at + 128 + q * 32, v);
#pragma unroll
            for (int e = 0; e < 32; ++e) sum[q * 32 + e] = k0 == 0 ? v[e] : sum[q * 32 + e] + v[e];
            tmem_load32(at + q * 32, v);
#pragma unroll
            for (int e = 0; e < 32; ++e) sum[q * 32 + e] += v[e];
          }
          release(acc);
        }
      }
#pragma unroll 1
      for (int h = 0; h < blocks; ++h) {
        if (!landed) break;
        const int64_t block = block0 + h * kBlockBytes;
        if (h > 0) load_old(t, block);
        if (t.op != kGram) {
          landed = !__any_sync(~0u, !mbar_wait(&old_full[warp], old_phase, kWaitPolls, abort, p.status));
          if (!landed) break;
          old_phase ^= 1;
        }
        __syncwarp();
        if (t.op == kGram) finish_block<kGram, SPLIT>(p, t, cb0 + h, row0, block, at + h * 64, sum, buf);
        else if (t.op == kSquare) finish_block<kSquare, SPLIT>(p, t, cb0 + h, row0, block, at + h * 64, sum, buf);
        else if (t.step + 1 < p.steps) finish_block<kApply, SPLIT>(p, t, cb0 + h, row0, block, at + h * 64, sum, buf);
        else finish_block<kApplyLast, SPLIT>(p, t, cb0 + h, row0, block, at + h * 64, sum, buf);
        if (h == 0) report(t.op != kApply || t.step + 1 < p.steps);  // (the last product leaves no bulk stores)
      }
      if (!landed) {  // winding down: a copy in flight still lands before the CTA goes
        if (t.op != kGram)
          for (uint32_t k = 0; k < kWaitPolls && !mbar_try_wait(&old_full[warp], old_phase); ++k) {
          }
        break;
      }
      if (!SPLIT) release((part - 1) & 1);
      report(false);
      owed = t.i;
    }
    report(false);
    if (lane == 0) bulk_wait_all();
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if (PAIR) cluster_sync();  // neither CTA goes while the other may still signal it or copy into it
  if (warp == EPI + 1) {
    fence_after();
    tmem_free<PAIR>(tmem);
  }
}

// How many CTAs (pairs of CTAs) of a product's kernel run at once on the
// current device; also lets the kernel use its shared memory.
template <class S>
cudaError_t resident(const void* kernel, int* workers) {
  static std::mutex mu;
  static std::vector<std::pair<int, int>> known;  // per device; one kernel has this shape
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  std::lock_guard<std::mutex> lock(mu);
  for (const auto& k : known)
    if (k.first == dev) {
      *workers = k.second;
      return cudaSuccess;
    }
  err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM + 1024);
  if (err != cudaSuccess) return err;
  *workers = device_sms();
  if (S::PAIR) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(device_sms() / S::CTAS * S::CTAS));
    cfg.blockDim = dim3(S::THREADS);
    cfg.dynamicSmemBytes = S::SMEM + 1024;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = S::CTAS;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    err = cudaOccupancyMaxActiveClusters(workers, kernel, &cfg);
    if (err != cudaSuccess) return err;
    if (*workers < 1) return cudaErrorInvalidConfiguration;
  }
  known.push_back({dev, *workers});
  return cudaSuccess;
}

}  // namespace

template <bool SPLIT, int CLUSTER>
cudaError_t launch_steps(OrthoTable& p, cudaStream_t stream) {
  using S = Shape<SPLIT, CLUSTER>;
  void (*kernel)(const OrthoTable) = steps_kernel<SPLIT, CLUSTER>;
  int workers = 0;
  const cudaError_t err = resident<S>(reinterpret_cast<const void*>(kernel), &workers);
  if (err != cudaSuccess) return err;
  int most = 0;
  for (int op = kGram; op <= kApply; ++op) {
    auto tiles = [&](const OrthoMat& m) { return tiles_of<S>(op, p.columns[op], m.mb, m.nb); };
    p.columns[op] = S::NU;
    fill_starts(p, op, tiles);
    if (S::NU > 1 && 2 * p.total[op] <= workers) {  // narrower tiles, so that more workers have one
      p.columns[op] = 1;
      fill_starts(p, op, tiles);
    }
    most = std::max(most, p.total[op]);
  }
  return launch_after(kernel, p, std::min(most, workers) * CLUSTER, S::THREADS,
                                             S::SMEM + 1024, CLUSTER, stream);
}

}  // namespace ar
