// What the kernels of the orthogonalised update share: their parameter table,
// the fp16 pairs that hold X, and launches.
#pragma once

#include "ortho.h"

#include <cuda.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "bulk.cuh"
#include "common.cuh"

namespace ar {

constexpr int kGroup = 64;  // matrices that run together
enum Op : int { kGram = 0, kSquare = 1, kApply = 2, kApplyLast = 3, kNone = 4 };

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

struct OrthoTable {
  CUtensorMap map;  // the workspace as rows of 128 bytes, boxes of 64 rows (pairs of CTAs)
  char* ws;
  StatusRef status;
  OrthoHyper hyper;
  float eps;
  int64_t part_off, sync_off;
  int n_mat, steps, out16;
  int total[3];     // work items: of the first kernels in total[0]; of a step's three products
  int columns[3];   // column blocks of 128 in a tile, per product
  OrthoMat mat[kGroup];
  OrthoIo io[kGroup];
  int32_t start[3][kGroup + 1];  // first work item of each matrix, per product
  OrthoPoly poly[kMaxOrthoSteps];
};

__device__ __forceinline__ int find_matrix(const OrthoTable& p, int item, int op = 0) {
  int lo = 0, hi = p.n_mat - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (p.start[op][mid] <= item) lo = mid;
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


inline cudaError_t launch_after(void (*kernel)(const OrthoTable), const OrthoTable& p, int grid, int threads, size_t smem,
                                int cluster, cudaStream_t stream) {
  if (grid <= 0) return cudaSuccess;
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

template <class F>
void fill_starts(OrthoTable& p, int op, F&& items) {
  int64_t n = 0;
  for (int i = 0; i < p.n_mat; ++i) {
    p.start[op][i] = int32_t(n);
    n += items(p.mat[i]);
  }
  p.start[op][p.n_mat] = int32_t(n);
  p.total[op] = int(n);
}

// The Newton-Schulz steps of a filled table (ortho_steps*.cu).
template <bool SPLIT, int CLUSTER>
cudaError_t launch_steps(OrthoTable& p, cudaStream_t stream);

}  // namespace ar
