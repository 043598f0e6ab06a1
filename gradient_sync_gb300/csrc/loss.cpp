// Host side of the losses: argument checks and launches (see include/ar.h).
#include <algorithm>
#include <cmath>
#include <new>
#include <utility>
#include <vector>

#include "internal.h"
#include "loss.h"

namespace {

using namespace ar;

constexpr double kLog2e = 1.4426950408889634074;

bool aligned(const void* p, size_t a) { return p != nullptr && reinterpret_cast<uintptr_t>(p) % a == 0; }
size_t esize(ar_dtype d) { return d == AR_BF16 ? 2 : 4; }

struct Range {
  uintptr_t lo, hi;
};
Range range(const void* p, int64_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return {a, a + uintptr_t(bytes > 0 ? bytes : 0)};
}
Range matrix_range(const void* p, int64_t rows, int64_t cols, int64_t ld, size_t es) {
  return range(p, rows > 0 ? ((rows - 1) * ld + cols) * int64_t(es) : 0);
}
bool overlap(Range a, Range b) { return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi; }

// Outputs must be apart from one another and from the inputs.
bool apart(const std::vector<Range>& outs, const std::vector<Range>& ins) {
  for (size_t i = 0; i < outs.size(); ++i) {
    for (size_t j = i + 1; j < outs.size(); ++j)
      if (overlap(outs[i], outs[j])) return false;
    for (const Range& r : ins)
      if (overlap(outs[i], r)) return false;
  }
  return true;
}

ar_status logits_params(const ar_logits* l, const float* logp, LossParams& p) {
  if (l == nullptr) return AR_EINVAL;
  if (l->rows < 0 || l->vocab < 1 || l->ld < l->vocab) return AR_EINVAL;
  if (l->dtype != AR_F32 && l->dtype != AR_BF16) return AR_EINVAL;
  if (!(l->temperature > 0.0f) || !std::isfinite(l->temperature)) return AR_EINVAL;
  const double k = kLog2e / double(l->temperature);
  if (!std::isfinite(float(k)) || !std::isfinite(1.0f / l->temperature)) return AR_EINVAL;
  if (l->rows >= (int64_t(1) << 31) || l->vocab > (int64_t(1) << 30)) return AR_EUNSUPPORTED;
  if (l->rows > 0 && l->ld > INT64_MAX / 8 / l->rows) return AR_EINVAL;
  if (l->rows > 0 && (!aligned(l->data, esize(l->dtype)) || !aligned(l->labels, 8) || !aligned(logp, 4)))
    return AR_EINVAL;
  p = LossParams{};
  p.x = l->data;
  p.rows = l->rows;
  p.vocab = l->vocab;
  p.ld = l->ld;
  p.labels = l->labels;
  p.k = float(k);
  p.inv_temp = float(1.0 / double(l->temperature));
  p.logp = const_cast<float*>(logp);
  return AR_OK;
}

// Checks shared by the two losses, and the parameters they have in common.
ar_status loss_params(const ar_logits* l, const float* logp, float* stats, void* d, int64_t dld, int64_t n_seq,
                      float denominator, float grad_scale, void* workspace, LossParams& p) {
  ar_status s = logits_params(l, logp, p);
  if (s != AR_OK) return s;
  if (!aligned(stats, 4) || !aligned(workspace, 16)) return AR_EINVAL;
  if (!std::isfinite(denominator) || denominator < 0.0f || !std::isfinite(grad_scale)) return AR_EINVAL;
  if (n_seq >= (int64_t(1) << 31)) return AR_EUNSUPPORTED;
  if (d != nullptr) {
    if (!aligned(d, esize(l->dtype)) || dld < l->vocab) return AR_EINVAL;
    if (p.rows > 0 && dld > INT64_MAX / 8 / p.rows) return AR_EINVAL;
  }
  p.d = d;
  p.dld = dld;
  p.n_seq = n_seq;
  p.denominator = denominator;
  p.grad_scale = grad_scale;
  p.stats = stats;
  const LossLayout w = loss_layout(p.rows, n_seq);
  char* base = static_cast<char*>(workspace);
  p.tickets = reinterpret_cast<unsigned int*>(base);
  p.seq_count = reinterpret_cast<int32_t*>(base + w.seq_count);
  p.row_a = reinterpret_cast<float*>(base + w.row_a);
  p.row_lse = reinterpret_cast<float2*>(base + w.row_lse);
  p.row_terms = reinterpret_cast<float*>(base + w.row_terms);
  return AR_OK;
}

// The call's outputs against one another and against its inputs; the gradient
// may be the logits' own memory.
bool loss_apart(const ar_logits* l, const LossParams& p, std::vector<Range> more_ins, std::vector<Range> more_outs) {
  const size_t es = esize(l->dtype);
  std::vector<Range> ins = std::move(more_ins), outs = std::move(more_outs);
  const Range x = matrix_range(p.x, p.rows, p.vocab, p.ld, es), d = matrix_range(p.d, p.d ? p.rows : 0, p.vocab, p.dld, es);
  ins.push_back(range(p.labels, 8 * p.rows));
  outs.push_back(range(p.logp, 4 * p.rows));
  outs.push_back(range(p.stats, 16));
  outs.push_back(range(p.tickets, loss_layout(p.rows, p.n_seq).bytes));
  const bool in_place = p.d == p.x && p.dld == p.ld;
  if (!in_place && overlap(x, d)) return false;
  for (const Range& o : outs)
    if (overlap(o, x)) return false;
  outs.push_back(d);
  return apart(outs, ins);
}

// Refuses while a device-side wait that ran out is recorded.
ar_status device_ready() {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return AR_ECUDA;
  volatile unsigned int* word = nullptr;
  if (host_status_word(dev, &word) != cudaSuccess) return AR_ECUDA;
  return *word != 0 ? AR_ETIMEOUT : AR_OK;
}

ar_status from_cuda(cudaError_t e) { return e == cudaSuccess ? AR_OK : AR_ECUDA; }

}  // namespace

extern "C" {

ar_status ar_loss_workspace(int64_t rows, int64_t n_seq, size_t* bytes) {
  if (bytes == nullptr || rows < 0 || n_seq < 0 || rows > INT64_MAX / 64 || n_seq > INT64_MAX / 64) return AR_EINVAL;
  *bytes = size_t(loss_layout(rows, n_seq).bytes);
  return AR_OK;
}

ar_status ar_token_logp(const ar_logits* logits, float* logp, void* stream) {
  LossParams p;
  ar_status s = logits_params(logits, logp, p);
  if (s != AR_OK || p.rows == 0) return s;
  const Range o = range(logp, 4 * p.rows);
  if (overlap(o, matrix_range(p.x, p.rows, p.vocab, p.ld, esize(logits->dtype))) ||
      overlap(o, range(p.labels, 8 * p.rows)))
    return AR_EINVAL;
  if ((s = device_ready()) != AR_OK) return s;
  return from_cuda(launch_token_logp(p, logits->dtype, static_cast<cudaStream_t>(stream)));
}

ar_status ar_policy_loss(const ar_logits* logits, const float* old_logp, const float* ref_logp,
                         const float* advantages, const int64_t* seq_start, int64_t n_seq, const ar_policy_desc* desc,
                         float* stats, float* logp, void* dlogits, int64_t dld, void* workspace, void* stream) try {
  if (desc == nullptr || n_seq < 1 || (seq_start == nullptr && n_seq != 1)) return AR_EINVAL;
  if (!(desc->clip_low >= 0.0f && desc->clip_low <= 1.0f) || !(desc->clip_high >= 0.0f) ||
      !std::isfinite(desc->clip_high) || !(desc->kl_coef >= 0.0f) || !std::isfinite(desc->kl_coef))
    return AR_EINVAL;
  if (desc->mean != AR_MEAN_TOKENS && desc->mean != AR_MEAN_SEQUENCES) return AR_EINVAL;
  LossParams p;
  ar_status s = loss_params(logits, logp, stats, dlogits, dld, n_seq, desc->denominator, desc->grad_scale, workspace, p);
  if (s != AR_OK) return s;
  if (desc->kl_coef > 0.0f && ref_logp == nullptr) return AR_EINVAL;
  if (p.rows > 0 && (!aligned(old_logp, 4) || !aligned(advantages, 4) || (ref_logp != nullptr && !aligned(ref_logp, 4))))
    return AR_EINVAL;
  if (seq_start != nullptr && !aligned(seq_start, 8)) return AR_EINVAL;
  std::vector<Range> ins = {range(old_logp, 4 * p.rows), range(advantages, 4 * p.rows)};
  if (ref_logp != nullptr) ins.push_back(range(ref_logp, 4 * p.rows));
  if (seq_start != nullptr) ins.push_back(range(seq_start, 8 * (n_seq + 1)));
  if (!loss_apart(logits, p, ins, {})) return AR_EINVAL;
  p.old_logp = old_logp;
  p.ref_logp = ref_logp;
  p.adv = advantages;
  p.lo = 1.0f - desc->clip_low;
  p.hi = 1.0f + desc->clip_high;
  p.kl = desc->kl_coef;
  p.seq_start = seq_start;
  p.by_sequence = desc->mean == AR_MEAN_SEQUENCES;
  if ((s = device_ready()) != AR_OK) return s;
  return from_cuda(launch_policy_loss(p, logits->dtype, static_cast<cudaStream_t>(stream)));
} catch (const std::bad_alloc&) {
  return AR_ENOMEM;
}

ar_status ar_preference_loss(const ar_logits* logits, const float* ref_logp, const int64_t* seq_start, int64_t n_seq,
                             const ar_preference_desc* desc, float* stats, float* ratios, float* logp, void* dlogits,
                             int64_t dld, void* workspace, void* stream) try {
  if (desc == nullptr || n_seq < 2 || n_seq % 2 != 0) return AR_EINVAL;
  if (!std::isfinite(desc->beta) || !std::isfinite(desc->target)) return AR_EINVAL;
  if (desc->form != AR_PREFER_SIGMOID && desc->form != AR_PREFER_SQUARE) return AR_EINVAL;
  if (!(desc->label_smoothing >= 0.0f && desc->label_smoothing <= 0.5f)) return AR_EINVAL;
  LossParams p;
  ar_status s = loss_params(logits, logp, stats, dlogits, dld, n_seq, desc->denominator, desc->grad_scale, workspace, p);
  if (s != AR_OK) return s;
  if (!aligned(seq_start, 8) || !aligned(ratios, 4) || (p.rows > 0 && !aligned(ref_logp, 4))) return AR_EINVAL;
  if (!loss_apart(logits, p, {range(ref_logp, 4 * p.rows), range(seq_start, 8 * (n_seq + 1))},
                  {range(ratios, 4 * n_seq)}))
    return AR_EINVAL;
  p.ref_logp = ref_logp;
  p.seq_start = seq_start;
  p.beta = desc->beta;
  p.smooth = desc->label_smoothing;
  p.target = desc->target;
  p.square = desc->form == AR_PREFER_SQUARE;
  p.normalize = desc->length_normalized != 0;
  p.ratios = ratios;
  if ((s = device_ready()) != AR_OK) return s;
  return from_cuda(launch_preference_loss(p, logits->dtype, static_cast<cudaStream_t>(stream)));
} catch (const std::bad_alloc&) {
  return AR_ENOMEM;
}

}  // extern "C"
