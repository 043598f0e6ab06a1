// Host side of the orthogonalised update: plans, argument checks and launches
// (see include/ar.h).
#include <algorithm>
#include <cmath>
#include <new>
#include <numeric>

#include "internal.h"
#include "ortho.h"

namespace {

using namespace ar;

constexpr int64_t kMaxDim = 1 << 20;
// Plans with at least this many 256 x 256 tiles of X run tiles of two CTAs,
// which read less per product but pad row blocks to 256 and have fewer tiles.
// Measured, one CTA against two: half precision 512 x 512 (4 tiles) 126 and
// 130 us, 1024 x 1024 (16) 169 and 162, 1536 x 1536 (36) 221 and 206,
// 1024 x 4096 (64) 271 and 247, 2048 x 4096 (128) 427 and 370; split 256 x 256
// (1) 149 and 140, 512 x 512 200 and 186, 1024 x 1024 (16) 284 and 233,
// 2048 x 4096 1004 and 743. (A matrix of at most 128 rows leaves a pair's second
// CTA without work, so that one tile alone stays with one CTA.)
constexpr int64_t kPairTiles = 16, kPairTilesSplit = 2;
constexpr float kDefault[3] = {3.4445f, -4.7750f, 2.0315f};

size_t esize(ar_dtype d) { return d == AR_BF16 ? 2 : 4; }
bool valid_dtype(ar_dtype d) { return d == AR_F32 || d == AR_BF16; }

// The polynomials of the steps, and whether they keep the operands in range:
// follows the singular values 0, 1/n, ..., 1 through all steps.
bool polynomials(const float* coef, int steps, std::vector<OrthoPoly>& out) {
  constexpr int kGrid = 4096;
  std::vector<double> s(kGrid + 1);
  for (int i = 0; i <= kGrid; ++i) s[i] = double(i) / kGrid;
  for (int k = 0; k < steps; ++k) {
    const float* q = coef != nullptr ? coef + 3 * k : kDefault;
    double lo = 0.0, hi = 0.0;
    // the values between grid points: the polynomials of all singular values
    // up to the largest one are bounded, not only of those that occur
    const double top = *std::max_element(s.begin(), s.end());
    for (int i = 0; i <= kGrid; ++i) {
      const double v = top * i / kGrid, l = v * v, b = double(q[1]) * l + double(q[2]) * l * l;
      lo = std::min(lo, b);
      hi = std::max(hi, b);
    }
    OrthoPoly p = {q[0], q[1], q[2], 0.0f};
    if (k >= steps - 2) p.t = float(-(lo + hi) / 2);
    if (std::max(std::fabs(lo), std::fabs(hi)) + std::fabs(p.t) > 12.0) return false;
    for (double& v : s) v = std::fabs(double(q[0]) * v + double(q[1]) * v * v * v + double(q[2]) * v * v * v * v * v);
    if (*std::max_element(s.begin(), s.end()) > 3.5) return false;
    out.push_back(p);
  }
  return true;
}

// Memory that a call reads or writes: `rows` rows of `width` bytes, `pitch` apart.
struct Range {
  uintptr_t lo, hi;
  uintptr_t pitch, width;
  bool write;
};
Range range(const ar_matrix& m, int64_t rows, int64_t cols, size_t es, bool write) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(m.data), pitch = uintptr_t(m.ld) * es, width = uintptr_t(cols) * es;
  return {a, a + uintptr_t(rows - 1) * pitch + width, pitch, width, write};
}

// Whether two overlapping ranges still share no byte: column windows of the
// same rows (a, with the lower start, and b), as the parts of a joint matrix are.
bool side_by_side(const Range& a, const Range& b) {
  if (a.pitch != b.pitch || a.pitch == 0) return false;
  const uintptr_t shift = (b.lo - a.lo) % a.pitch;
  return shift >= a.width && shift + b.width <= a.pitch;
}

// No written range overlaps another one.
bool apart(std::vector<Range> v) {
  std::sort(v.begin(), v.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
  std::vector<Range> open;
  for (const Range& r : v) {
    open.erase(std::remove_if(open.begin(), open.end(), [&](const Range& o) { return o.hi <= r.lo; }), open.end());
    for (const Range& o : open)
      if ((o.write || r.write) && !side_by_side(o, r)) return false;
    open.push_back(r);
  }
  return true;
}

bool valid(const ar_matrix& m, int64_t cols, size_t es) {
  return m.data != nullptr && reinterpret_cast<uintptr_t>(m.data) % es == 0 && m.ld >= cols && m.ld <= INT64_MAX / 8 / kMaxDim;
}

// Whether every access to rows of `cols` elements can be 16 bytes wide, `step` elements at a time.
bool wide(const void* p, int64_t ld, int64_t step) {
  return p == nullptr || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % step == 0);
}
void set_access(OrthoIo& q, int64_t cols, size_t out_size) {
  q.flat = q.g_ld == cols && (q.m == nullptr || (q.m_ld == cols && q.m_out_ld == cols));
  q.vec_in = cols % 8 == 0 && wide(q.g, q.g_ld, 8) && wide(q.m, q.m_ld, 8) && wide(q.m_out, q.m_out_ld, 8);
  const int64_t step = int64_t(16 / out_size);
  q.vec_out = wide(q.w, q.w_ld, step) && wide(q.w_out, q.w_out_ld, step);
}

bool same(const ar_matrix& a, const ar_matrix& b) { return a.data == b.data && a.ld == b.ld; }

ar_status guard(const void* workspace) {
  if (workspace == nullptr || reinterpret_cast<uintptr_t>(workspace) % 16 != 0) return AR_EINVAL;
  return AR_OK;
}

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

ar_status ar_ortho_plan(const ar_ortho_desc* desc, ar_ortho_plan_t** out) try {
  if (desc == nullptr || out == nullptr) return AR_EINVAL;
  *out = nullptr;
  const int n = desc->n_matrices;
  if (n < 1 || desc->rows == nullptr || desc->cols == nullptr) return AR_EINVAL;
  if (!valid_dtype(desc->in_dtype) || !valid_dtype(desc->out_dtype)) return AR_EINVAL;
  if (desc->steps < 1 || desc->steps > AR_MAX_ORTHO_STEPS) return AR_EINVAL;
  if (!(desc->eps >= 0.0f) || !std::isfinite(desc->eps)) return AR_EINVAL;
  if (desc->precision < AR_PRECISION_AUTO || desc->precision > AR_PRECISION_SPLIT) return AR_EINVAL;
  if (n > AR_MAX_MATRICES) return AR_EUNSUPPORTED;
  for (int i = 0; i < n; ++i)
    if (desc->rows[i] < 1 || desc->cols[i] < 1 || desc->rows[i] > kMaxDim || desc->cols[i] > kMaxDim) return AR_EINVAL;
  if (desc->coefficients != nullptr)
    for (int i = 0; i < 3 * desc->steps; ++i)
      if (!std::isfinite(desc->coefficients[i])) return AR_EINVAL;
  ar_ortho_plan_t p = {};
  if (!polynomials(desc->coefficients, desc->steps, p.poly)) return AR_EUNSUPPORTED;
  p.in_dtype = desc->in_dtype;
  p.out_dtype = desc->out_dtype;
  p.eps = desc->eps;
  p.split = desc->precision == AR_PRECISION_SPLIT || (desc->precision == AR_PRECISION_AUTO && desc->out_dtype == AR_F32);
  int64_t work = 0;
  for (int i = 0; i < n; ++i) {
    const int64_t r = desc->rows[i], c = desc->cols[i], mb = (std::min(r, c) + 127) / 128, nb = (std::max(r, c) + 127) / 128;
    work += (mb + 1) / 2 * ((nb + 1) / 2);
  }
  p.cluster = work >= (p.split ? kPairTilesSplit : kPairTiles) ? 2 : 1;
  int64_t at = 0, parts = 0, blocks = 0;
  for (int i = 0; i < n; ++i) {
    const int64_t r = desc->rows[i], c = desc->cols[i];
    OrthoMat m = {};
    m.turned = r > c;
    m.m = int32_t(std::min(r, c));
    m.n = int32_t(std::max(r, c));
    m.mb = (m.m + 127) / 128;
    if (p.cluster > 1) m.mb += m.mb % 2;
    m.nb = (m.n + 127) / 128 * 2;
    // entries of X have rms up to 1 / sqrt(n): held as about 16
    m.sx = std::ldexp(16.0f, int(std::ceil(std::log2(double(m.n)) / 2)));
    m.x_bytes = int64_t(m.mb) * m.nb * kBlockBytes;
    m.a_bytes = int64_t(m.mb) * (2 * m.mb) * kBlockBytes;
    m.x = at;
    m.a = at + 4 * m.x_bytes;
    at = m.a + (p.split ? 4 : 2) * m.a_bytes;
    m.part = int32_t(parts);
    m.n_part = int32_t((int64_t(m.m) * m.n + kOrthoChunk - 1) / kOrthoChunk);
    parts += m.n_part;
    blocks += int64_t(m.mb) * m.nb;
    if (blocks > INT32_MAX / 2 || parts > INT32_MAX / 2) return AR_EUNSUPPORTED;
    p.mats.push_back(m);
    p.rows.push_back(r);
    p.cols.push_back(c);
  }
  if (at / 128 > INT32_MAX) return AR_EUNSUPPORTED;
  p.part_off = at;
  p.sync_off = at + 8 * parts;
  p.bytes = at + (8 * parts + 4 * (1 + n) + 255) / 256 * 256;
  p.order.resize(n);
  std::iota(p.order.begin(), p.order.end(), 0);
  std::stable_sort(p.order.begin(), p.order.end(), [&](int a, int b) { return p.mats[a].nb > p.mats[b].nb; });
  *out = new ar_ortho_plan_t(std::move(p));
  return AR_OK;
} catch (const std::bad_alloc&) {
  return AR_ENOMEM;
}

void ar_ortho_plan_destroy(ar_ortho_plan_t* plan) { delete plan; }

ar_status ar_ortho_workspace(const ar_ortho_plan_t* plan, size_t* bytes) {
  if (plan == nullptr || bytes == nullptr) return AR_EINVAL;
  *bytes = size_t(plan->bytes);
  return AR_OK;
}

ar_status ar_orthogonalize(const ar_ortho_plan_t* plan, const ar_matrix* in, const ar_matrix* out, void* workspace,
                           void* stream) try {
  if (plan == nullptr || in == nullptr || out == nullptr || guard(workspace) != AR_OK) return AR_EINVAL;
  const int n = int(plan->mats.size());
  const size_t ie = esize(plan->in_dtype), oe = esize(plan->out_dtype);
  std::vector<Range> ranges = {{uintptr_t(workspace), uintptr_t(workspace) + uintptr_t(plan->bytes), 0, 0, true}};
  std::vector<OrthoIo> io(n);
  for (int i = 0; i < n; ++i) {
    const int64_t r = plan->rows[i], c = plan->cols[i];
    if (!valid(in[i], c, ie) || !valid(out[i], c, oe)) return AR_EINVAL;
    if (!(same(in[i], out[i]) && ie == oe)) ranges.push_back(range(in[i], r, c, ie, false));
    ranges.push_back(range(out[i], r, c, oe, true));
    io[i] = OrthoIo{};
    io[i].g = in[i].data;
    io[i].g_ld = in[i].ld;
    io[i].w_out = out[i].data;
    io[i].w_out_ld = out[i].ld;
    io[i].alpha = 1.0f;
    set_access(io[i], c, oe);
  }
  if (!apart(std::move(ranges))) return AR_EINVAL;
  const ar_status s = device_ready();
  if (s != AR_OK) return s;
  const OrthoHyper hyper = {0.0f, 1.0f, 1.0f, 0, 0, nullptr};
  return from_cuda(launch_ortho(*plan, io.data(), hyper, static_cast<char*>(workspace), static_cast<cudaStream_t>(stream)));
} catch (const std::bad_alloc&) {
  return AR_ENOMEM;
}

ar_status ar_muon_step(const ar_ortho_plan_t* plan, const ar_muon_desc* desc, const ar_matrix* params,
                       const ar_matrix* grads, const ar_matrix* momenta, const ar_matrix* params_out,
                       const ar_matrix* momenta_out, void* workspace, void* stream) {
  return ar_muon_step_clipped(plan, desc, params, grads, momenta, params_out, momenta_out, nullptr, workspace, stream);
}

ar_status ar_muon_step_clipped(const ar_ortho_plan_t* plan, const ar_muon_desc* desc, const ar_matrix* params,
                               const ar_matrix* grads, const ar_matrix* momenta, const ar_matrix* params_out,
                               const ar_matrix* momenta_out, const float* clip, void* workspace, void* stream) try {
  if (plan == nullptr || desc == nullptr || params == nullptr || grads == nullptr || momenta == nullptr ||
      guard(workspace) != AR_OK)
    return AR_EINVAL;
  if (!std::isfinite(desc->lr) || !std::isfinite(desc->momentum) || !std::isfinite(desc->weight_decay) ||
      !std::isfinite(desc->grad_scale) || desc->adjust < AR_ADJUST_NONE || desc->adjust > AR_ADJUST_RMS)
    return AR_EINVAL;
  if (clip != nullptr && reinterpret_cast<uintptr_t>(clip) % 4 != 0) return AR_EINVAL;
  if (params_out == nullptr) params_out = params;
  if (momenta_out == nullptr) momenta_out = momenta;
  const int n = int(plan->mats.size());
  const size_t ge = esize(plan->in_dtype), we = esize(plan->out_dtype);
  std::vector<Range> ranges = {{uintptr_t(workspace), uintptr_t(workspace) + uintptr_t(plan->bytes), 0, 0, true}};
  std::vector<OrthoIo> io(n);
  for (int i = 0; i < n; ++i) {
    const int64_t r = plan->rows[i], c = plan->cols[i];
    if (!valid(params[i], c, we) || !valid(grads[i], c, ge) || !valid(momenta[i], c, 4) || !valid(params_out[i], c, we) ||
        !valid(momenta_out[i], c, 4))
      return AR_EINVAL;
    ranges.push_back(range(grads[i], r, c, ge, false));
    if (!same(params[i], params_out[i])) ranges.push_back(range(params[i], r, c, we, false));
    if (!same(momenta[i], momenta_out[i])) ranges.push_back(range(momenta[i], r, c, 4, false));
    ranges.push_back(range(params_out[i], r, c, we, true));
    ranges.push_back(range(momenta_out[i], r, c, 4, true));
    OrthoIo& q = io[i];
    q = OrthoIo{};
    q.g = grads[i].data;
    q.g_ld = grads[i].ld;
    q.m = static_cast<const float*>(momenta[i].data);
    q.m_ld = momenta[i].ld;
    q.m_out = static_cast<float*>(momenta_out[i].data);
    q.m_out_ld = momenta_out[i].ld;
    q.w = params[i].data;
    q.w_ld = params[i].ld;
    q.w_out = params_out[i].data;
    q.w_out_ld = params_out[i].ld;
    const double rows = double(r), cols = double(c);
    const double adjust = desc->adjust == AR_ADJUST_SHAPE ? std::sqrt(std::max(1.0, rows / cols))
                          : desc->adjust == AR_ADJUST_RMS ? 0.2 * std::sqrt(std::max(rows, cols))
                                                          : 1.0;
    q.alpha = float(-double(desc->lr) * adjust);
    set_access(q, c, we);
  }
  if (clip != nullptr) ranges.push_back({uintptr_t(clip), uintptr_t(clip) + 16, 0, 0, false});
  if (!apart(std::move(ranges))) return AR_EINVAL;
  const ar_status s = device_ready();
  if (s != AR_OK) return s;
  const OrthoHyper hyper = {desc->momentum, desc->grad_scale, float(1.0 - double(desc->lr) * double(desc->weight_decay)), 1,
                            desc->nesterov != 0, clip};
  return from_cuda(launch_ortho(*plan, io.data(), hyper, static_cast<char*>(workspace), static_cast<cudaStream_t>(stream)));
} catch (const std::bad_alloc&) {
  return AR_ENOMEM;
}

}  // extern "C"
