// Declarations shared by the host side of the losses (loss.cpp) and their
// kernels (loss.cu). Not part of the public ABI.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/ar.h"

namespace ar {

enum LossMode : int { kLogp = 0, kPolicy = 1, kPrefForward = 2, kPrefBackward = 3 };

struct LossParams {
  const void* x;          // logits, row t at x + t * ld
  int64_t rows, vocab, ld;
  const int64_t* labels;  // < 0: the row is not part of the loss
  float k;                // log2(e) / temperature
  float inv_temp;
  float* logp;            // [rows]
  void* d;                // gradient of the logits, row t at d + t * dld; null: none
  int64_t dld;
  // policy loss
  const float* old_logp;
  const float* ref_logp;  // null: no KL term
  const float* adv;
  float lo, hi, kl;       // clip bounds 1 - low, 1 + high; KL coefficient
  // sequences
  const int64_t* seq_start;  // null: one sequence of all rows
  int64_t n_seq;
  int by_sequence;        // weights 1 / labelled tokens of the sequence (else 1)
  float denominator;      // > 0: replaces the counted one
  float grad_scale;
  // preference loss
  float beta, smooth, target;
  int square, normalize;
  float* ratios;          // [n_seq]
  float* stats;           // [4]
  // workspace
  unsigned int* tickets;  // [0]: pairs done
  int32_t* seq_count;     // [n_seq] labelled tokens
  float* row_a;           // [rows] policy: weight before the total; preference: coefficient
  int cluster;            // CTAs a row
  int few;                // a few rows: weights and pairs are worked out by the rows' kernels
  unsigned int* status_word;         // where waits that ran out are recorded
  unsigned int* const* status_host;
  float2* row_lse;        // [rows] preference: (base-2 shift, 1 / sum)
  float* row_terms;       // policy: [3 * rows] weighted loss terms;
                          // preference: [rows] log ratios, then [4 * pairs] terms
};

// Byte offsets of the workspace's parts, and its size.
struct LossLayout {
  int64_t seq_count, row_a, row_lse, row_terms, bytes;
};
inline LossLayout loss_layout(int64_t rows, int64_t n_seq) {
  auto up = [](int64_t v) { return (v + 255) / 256 * 256; };
  LossLayout l;
  l.seq_count = 256;  // tickets come first
  l.row_a = l.seq_count + up(4 * n_seq);
  l.row_lse = l.row_a + up(4 * rows);
  l.row_terms = l.row_lse + up(8 * rows);
  const int64_t terms = rows + (2 * rows > 2 * n_seq ? 2 * rows : 2 * n_seq);
  l.bytes = l.row_terms + up(4 * terms);
  return l;
}

cudaError_t launch_token_logp(const LossParams& p, ar_dtype dtype, cudaStream_t stream);
cudaError_t launch_policy_loss(const LossParams& p, ar_dtype dtype, cudaStream_t stream);
cudaError_t launch_preference_loss(const LossParams& p, ar_dtype dtype, cudaStream_t stream);

}  // namespace ar
