// Declarations shared by the host side of the orthogonalised update
// (ortho.cpp) and its kernels (ortho.cu). Not part of the public ABI.
#pragma once

#include <cstdint>
#include <vector>

#include <cuda_runtime.h>

#include "../../include/ar.h"

namespace ar {

constexpr int kMaxOrthoSteps = 16;
constexpr int64_t kOrthoChunk = 32768;  // elements per partial sum of squares
constexpr int64_t kBlockBytes = 16384;  // one block: 128 rows x 64 columns of fp16

// One matrix as the kernels hold it: X has m = min(rows, cols) rows and
// n = max(rows, cols) columns (a tall matrix is held transposed), padded with
// zeros to `mb` row blocks of 128 and `nb` column blocks of 64 (nb even).
struct OrthoMat {
  int32_t m, n, mb, nb;
  int32_t turned;
  float sx;           // X is held times this power of two
  int64_t x;          // workspace offset: X of even steps hi, lo, of odd steps hi, lo
  int64_t a;          // workspace offset: A hi, (A lo), B hi, (B lo)
  int64_t x_bytes, a_bytes;
  int32_t part, n_part;  // partial sums of squares
};

// What a call reads and writes for one matrix.
struct OrthoIo {
  const void* g;   // input or gradient
  const float* m;  // momentum
  float* m_out;
  const void* w;   // weights (null: the result itself is wanted)
  void* w_out;
  int64_t g_ld, m_ld, m_out_ld, w_ld, w_out_ld;
  float alpha;     // factor of the orthogonal matrix in the result
  bool flat;       // g, m and m_out are contiguous: element e of the matrix is element e of each
  bool vec_in;     // g, m and m_out can be read eight elements at a time
  bool vec_out;    // w and w_out can be accessed 16 bytes at a time
};

struct OrthoHyper {
  float mu, grad_scale, keep;  // keep: 1 - lr * weight decay
  int muon, nesterov;
  const float* clip;  // statistics of a gradient norm (null: none): [1] multiplies gradients too, [3] = 0: they count as 0
};

struct OrthoPoly {
  float a, b, c, t;  // X <- (a - t) X + (b A + c A A + t I) X
};

}  // namespace ar

struct ar_ortho_plan {
  std::vector<ar::OrthoMat> mats;  // in the caller's order
  std::vector<int64_t> rows, cols;
  std::vector<int> order;          // launch order: longest products first
  std::vector<ar::OrthoPoly> poly; // one per step
  ar_dtype in_dtype, out_dtype;
  float eps;
  bool split;
  int cluster;  // CTAs that work on a tile together: 1, or 2 (row blocks padded to an even number)
  int64_t part_off, sync_off, bytes;  // partial sums of squares; the products' counters
};

namespace ar {

cudaError_t launch_ortho(const ar_ortho_plan_t& plan, const OrthoIo* io, const OrthoHyper& hyper, char* ws,
                         cudaStream_t stream);

}  // namespace ar
