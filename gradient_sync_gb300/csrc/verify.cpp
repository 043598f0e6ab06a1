// Host side of the verification of drafted tokens: argument checks and launches
// (see include/ar.h).
#include <cmath>
#include <vector>

#include "internal.h"
#include "verify.h"

namespace {

using namespace ar;

constexpr double kLog2e = 1.4426950408889634074;

bool aligned(const void* p, size_t a) { return p != nullptr && reinterpret_cast<uintptr_t>(p) % a == 0; }

struct Range {
  uintptr_t lo, hi;
};
Range range(const void* p, int64_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return {a, a + uintptr_t(p != nullptr && bytes > 0 ? bytes : 0)};
}
bool overlap(const Range& a, const Range& b) { return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi; }

ar_status score_rows(const ar_score_rows& r, int64_t rows, int64_t vocab, VerifyRows& out, Range& memory) {
  if (r.rows != rows || r.ld < vocab) return AR_EINVAL;
  if (r.dtype != AR_F32 && r.dtype != AR_BF16) return AR_EINVAL;
  if (!(r.temperature > 0.0f) || !std::isfinite(r.temperature)) return AR_EINVAL;
  const double k = kLog2e / double(r.temperature);
  if (!std::isfinite(float(k)) || !std::isfinite(1.0f / r.temperature)) return AR_EINVAL;
  const int64_t es = r.dtype == AR_BF16 ? 2 : 4;
  if (rows > 0 && (!aligned(r.data, size_t(es)) || r.ld > INT64_MAX / 8 / rows)) return AR_EINVAL;
  out.data = static_cast<const char*>(r.data);
  out.ld = r.ld;
  out.bf16 = r.dtype == AR_BF16;
  out.k = float(k);
  memory = range(r.data, rows > 0 ? ((rows - 1) * r.ld + vocab) * es : 0);
  return AR_OK;
}

ar_status device_ready() {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return AR_ECUDA;
  volatile unsigned int* word = nullptr;
  if (host_status_word(dev, &word) != cudaSuccess) return AR_ECUDA;
  return *word != 0 ? AR_ETIMEOUT : AR_OK;
}

ar_status sizes_ok(int64_t n_drafts, int64_t n_seq, int64_t vocab) {
  if (n_drafts < 0 || n_seq < 1 || vocab < 1) return AR_EINVAL;
  const int64_t most = int64_t(1) << 31;
  if (n_drafts >= most || n_seq >= most || n_drafts + n_seq >= most || vocab > (int64_t(1) << 30)) return AR_EUNSUPPORTED;
  return AR_OK;
}

}  // namespace

extern "C" {

ar_status ar_verify_workspace(int64_t n_drafts, int64_t n_seq, int64_t vocab, size_t* bytes) {
  if (bytes == nullptr) return AR_EINVAL;
  const ar_status s = sizes_ok(n_drafts, n_seq, vocab);
  if (s == AR_OK) *bytes = size_t(verify_layout(n_drafts, n_seq).bytes);
  return s;
}

ar_status ar_verify_drafts(const ar_verify_desc* d, int64_t* accepted, int64_t* tokens, float* logp, void* workspace,
                           void* stream) {
  if (d == nullptr) return AR_EINVAL;
  ar_status s = sizes_ok(d->n_drafts, d->n_seq, d->vocab);
  if (s != AR_OK) return s;
  if (d->mode != AR_VERIFY_SAMPLE && d->mode != AR_VERIFY_GREEDY) return AR_EINVAL;
  const bool greedy = d->mode == AR_VERIFY_GREEDY;
  const int64_t rows = d->n_drafts + d->n_seq;
  VerifyParams p = {};
  Range x = {0, 0}, y = {0, 0};
  if ((s = score_rows(d->target, rows, d->vocab, p.target, x)) != AR_OK) return s;
  if (d->draft.data != nullptr && d->n_drafts > 0) {
    if (greedy) return AR_EINVAL;
    if ((s = score_rows(d->draft, d->n_drafts, d->vocab, p.draft, y)) != AR_OK) return s;
  }
  if ((d->n_drafts > 0 && !aligned(d->drafts, 8)) || (!greedy && !aligned(d->uniforms, 4))) return AR_EINVAL;
  if (d->draft_start == nullptr ? d->n_seq != 1 : !aligned(d->draft_start, 8)) return AR_EINVAL;
  if (!aligned(accepted, 8) || !aligned(tokens, 8) || !aligned(logp, 4) || !aligned(workspace, 16)) return AR_EINVAL;
  const VerifyLayout layout = verify_layout(d->n_drafts, d->n_seq);
  const Range outs[] = {range(accepted, 8 * d->n_seq), range(tokens, 8 * rows), range(logp, 4 * rows),
                        range(workspace, layout.bytes)};
  const Range ins[] = {x, y, range(d->drafts, 8 * d->n_drafts), range(greedy ? nullptr : d->uniforms, 4 * rows),
                       range(d->draft_start, 8 * (d->n_seq + 1))};
  for (int i = 0; i < 4; ++i) {
    for (int j = i + 1; j < 4; ++j)
      if (overlap(outs[i], outs[j])) return AR_EINVAL;
    for (const Range& r : ins)
      if (overlap(outs[i], r)) return AR_EINVAL;
  }
  p.vocab = d->vocab;
  p.drafts = d->drafts;
  p.uniforms = d->uniforms;
  p.draft_start = d->draft_start;
  p.n_drafts = d->n_drafts;
  p.n_seq = d->n_seq;
  p.greedy = greedy;
  p.accepted = accepted;
  p.tokens = tokens;
  p.logp = logp;
  char* base = static_cast<char*>(workspace);
  p.sums = reinterpret_cast<RowSums*>(base);
  p.done = reinterpret_cast<int32_t*>(base + layout.done);
  p.fallen = reinterpret_cast<int32_t*>(base + layout.fallen);
  if ((s = device_ready()) != AR_OK) return s;
  return launch_verify(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? AR_OK : AR_ECUDA;
}

}  // extern "C"
