// Declarations shared by the host side of the gradient norm, clipping and AdamW
// (grads.cpp) and their kernels (grads.cu). Not part of the public ABI.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/ar.h"

namespace ar {

// Tensors of one launch: their table is a kernel argument (at most 32764 bytes
// of those), so that neither a copy nor device memory of its own is needed and
// a captured launch is complete in itself. Short lists take a short table.
constexpr int kGradCap = 768, kGradCapSmall = 48;
constexpr int kAdamCap = 360, kAdamCapSmall = 40;
constexpr int kMaxGradCtas = 512;  // CTAs of a norm launch

struct GradEntry {
  const char* in;
  char* out;      // clipping only
  int64_t first;  // granules (16 aligned bytes, and some a tensor) of the tensors before this one
  int64_t count;  // elements * 2 + (1: bf16)
};

template <int CAP>
struct GradTable {
  int n;
  int64_t granules;  // of all entries
  int64_t per;       // of them a warp
  int64_t keep;      // of those, the last ones that stay in the L2
  GradEntry e[CAP];
};

// What the launches of one call have in common.
struct GradJob {
  int kind;  // ar_norm_kind
  float max_norm, max_norm_low, eps, eps_low;  // each as two numbers
  float grad_scale;
  float* stats;
  float* norms;    // may be null
  void* groups;    // workspace: the sum (or maximum) of every launch's tensors, 12 bytes each
  void* partials;  // workspace: those of one launch's CTAs, [CTAs + tensors]
};

// Byte offsets of the workspace's parts, and its size.
constexpr int kGradGroups = (AR_MAX_TENSORS + kGradCap - 1) / kGradCap;
constexpr int64_t kGradPartials = (12 * kGradGroups + 255) / 256 * 256;
constexpr int64_t kGradWorkspace = kGradPartials + (12 * (kMaxGradCtas + kGradCap) + 255) / 256 * 256;

// A tensor of a call, as checked.
struct GradTensor {
  const char* in;
  char* out;
  int64_t count;
  bool bf16;
};

struct AdamEntry {
  const void* g;
  const void* w;  // weights: the master, or the parameter
  const float* m;
  const float* v;
  void* w_out;
  void* p_out;  // the parameter beside a master; else null
  float* m_out;
  float* v_out;
  int64_t count;
  int32_t first;   // tiles of the tensors before this one
  uint8_t g_bf16, w_bf16, p_bf16;
  uint8_t phase;   // elements between a multiple of 8 and the first one, alike in all arrays; 255: not alike
};

template <int CAP>
struct AdamTable {
  int n;
  int tiles;
  AdamEntry e[CAP];
};

struct AdamRates {
  float beta1, beta2, rest1, rest2;  // rest = 1 - beta
  float rate;                        // lr / (1 - beta1^t)
  float inv_root;                    // 1 / sqrt(1 - beta2^t)
  float eps, keep;                   // keep = 1 - lr * weight_decay
};

struct AdamJob {
  AdamRates rates;             // for a step and a learning rate that the host knows
  const int64_t* device_step;  // null: it does
  const float* device_lr;      // null: it does
  int64_t step;                // for those that it does not
  float lr, weight_decay, log1, log1_low, log2, log2_low;  // log beta as two numbers
  const float* clip;           // null: none
  float grad_scale;
  bool in_place;               // every output is its input
};

constexpr int kAdamTile = 4096;  // elements

cudaError_t launch_grad_norm(const GradTensor* t, int n, bool clip, const GradJob& job, cudaStream_t stream);
cudaError_t launch_adamw(const AdamEntry* e, int n, const AdamJob& job, cudaStream_t stream);

}  // namespace ar
