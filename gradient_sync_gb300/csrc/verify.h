// Declarations shared by the host side of the verification of drafted tokens
// (verify.cpp) and its kernels (verify.cu). Not part of the public ABI.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/ar.h"

namespace ar {

// A part of a row's sums: shift and sum of the target's and of the draft's, or, greedy,
// of the target's, its largest score and that one's place.
struct RowSums {
  float v[4];
};
constexpr int kVerifyPartBits = 5;  // at most 32 parts of a row

struct VerifyRows {
  const char* data;
  int64_t ld;
  int bf16;
  float k;  // log2(e) / temperature
};

struct VerifyParams {
  VerifyRows target, draft;  // draft.data null: no distributions
  int64_t vocab;
  const int64_t* drafts;
  const float* uniforms;
  const int64_t* draft_start;  // null: one sequence
  int64_t n_drafts, n_seq;
  int greedy;
  int64_t* accepted;
  int64_t* tokens;
  float* logp;
  RowSums* sums;    // workspace, [n_drafts + n_seq][parts]
  int32_t* done;    // workspace, [n_drafts + n_seq]: parts of a row that are
  int32_t* fallen;  // workspace, [n_seq]: a draft that fell, by its place; null: not kept
  int parts, part_bits;  // of a row in sums_kernel: a power of two
  int pitch;             // rows that are visited one after the other
  int rank_bits;         // CTAs a sequence in draw_kernel: a power of two
};

// Byte offsets of the workspace's parts, and its size.
struct VerifyLayout {
  int64_t done, fallen, bytes;
};
inline VerifyLayout verify_layout(int64_t n_drafts, int64_t n_seq) {
  const auto up = [](int64_t v) { return (v + 255) / 256 * 256; };
  VerifyLayout l;
  l.done = (int64_t(sizeof(RowSums)) << kVerifyPartBits) * (n_drafts + n_seq);
  l.fallen = l.done + up(4 * (n_drafts + n_seq));
  l.bytes = l.fallen + up(4 * n_seq);
  return l;
}

cudaError_t launch_verify(const VerifyParams& p, cudaStream_t stream);

}  // namespace ar
