// Declarations shared by the host side of the verification of drafted tokens
// (verify.cpp) and its kernels (verify.cu). Not part of the public ABI.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/ar.h"

namespace ar {

// What a row's CTA leaves for the sequence: whether its draft stands, the
// token drawn in its place, and the log-probabilities of both.
struct RowResult {
  int64_t token;
  float token_logp, draft_logp;
  int32_t stands;
  int32_t unused;
};

struct VerifyRows {
  const char* data;
  int64_t ld;
  int bf16;
  double inv_temp;
  float k, k_low;  // log2(e) / temperature, and what fp32 leaves of it
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
  RowResult* results;  // workspace, [n_drafts + n_seq]
  int32_t* fallen;     // workspace, [n_seq]: a draft that fell, by its place; null: not kept
  int ranks;           // CTAs a row
  int64_t pitch;       // rows are visited this far apart
  unsigned int* status_word;  // where waits that ran out are recorded
  unsigned int* const* status_host;
};

// Byte offset of `fallen` in the workspace, and its size.
inline int64_t verify_fallen(int64_t n_drafts, int64_t n_seq) {
  return (int64_t(sizeof(RowResult)) * (n_drafts + n_seq) + 255) / 256 * 256;
}
inline int64_t verify_bytes(int64_t n_drafts, int64_t n_seq) {
  return verify_fallen(n_drafts, n_seq) + (4 * n_seq + 255) / 256 * 256;
}

cudaError_t launch_verify(const VerifyParams& p, cudaStream_t stream);

}  // namespace ar
