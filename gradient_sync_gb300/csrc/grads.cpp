// Host side of the gradient norm, clipping and AdamW: argument checks and
// launches (see include/ar.h).
#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "grads.h"
#include "internal.h"

namespace {

using namespace ar;

constexpr int64_t kMaxCount = int64_t(1) << 40;

int64_t esize(ar_dtype d) { return d == AR_BF16 ? 2 : 4; }
bool aligned(const void* p, size_t a) { return p != nullptr && reinterpret_cast<uintptr_t>(p) % a == 0; }

bool valid(const ar_tensor& t) {
  if (t.count < 0 || t.count > kMaxCount || (t.dtype != AR_F32 && t.dtype != AR_BF16)) return false;
  return t.count == 0 || aligned(t.data, size_t(esize(t.dtype)));
}
bool valid(const ar_tensor* t, int n) {
  return t != nullptr && std::all_of(t, t + n, [](const ar_tensor& v) { return valid(v); });
}

// Memory that a call reads or writes.
struct Range {
  uintptr_t lo, hi;
  bool write;
};
Range range(const void* p, int64_t bytes, bool write) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return {a, a + uintptr_t(bytes), write};
}
Range range(const ar_tensor& t, bool write) { return range(t.data, t.count * esize(t.dtype), write); }

// The ranges of a call, list by list. Lists are mostly in the order of their
// addresses, so that merging them is quicker than sorting all ranges.
struct Ranges {
  std::vector<Range> v;
  std::vector<size_t> ends;  // of ascending runs
  explicit Ranges(size_t most) { v.reserve(most); }
  void add(const Range& r) {
    if (r.lo >= r.hi) return;
    if (!v.empty() && r.lo < v.back().lo) ends.push_back(v.size());
    v.push_back(r);
  }
  // Whether no written range overlaps another one.
  bool apart() {
    const auto by_lo = [](const Range& a, const Range& b) { return a.lo < b.lo; };
    ends.push_back(v.size());
    if (ends.size() > 64) {
      std::sort(v.begin(), v.end(), by_lo);
    } else {
      while (ends.size() > 1) {
        size_t from = 0, kept = 0;
        for (size_t i = 0; i < ends.size(); i += 2) {
          if (i + 1 < ends.size()) {
            std::inplace_merge(v.begin() + from, v.begin() + ends[i], v.begin() + ends[i + 1], by_lo);
            from = ends[i + 1];
          } else {
            from = ends[i];
          }
          ends[kept++] = from;
        }
        ends.resize(kept);
      }
    }
    uintptr_t written = 0, any = 0;  // the ends so far
    for (const Range& r : v) {
      if (r.lo < written || (r.write && r.lo < any)) return false;
      any = std::max(any, r.hi);
      if (r.write) written = std::max(written, r.hi);
    }
    return true;
  }
};

// A number as two of fp32.
void halves(double v, float& hi, float& low) {
  hi = float(v);
  low = std::isfinite(hi) ? float(v - double(hi)) : 0.0f;
}

ar_status device_ready() {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return AR_ECUDA;
  volatile unsigned int* word = nullptr;
  if (host_status_word(dev, &word) != cudaSuccess) return AR_ECUDA;
  return *word != 0 ? AR_ETIMEOUT : AR_OK;
}

ar_status from_cuda(cudaError_t e) { return e == cudaSuccess ? AR_OK : AR_ECUDA; }

ar_status count_ok(int n) { return n < 1 ? AR_EINVAL : n > AR_MAX_TENSORS ? AR_EUNSUPPORTED : AR_OK; }

ar_status grad_norm(const ar_tensor* grads, int n, const ar_tensor* outs, bool clip, const ar_norm_desc* desc,
                    float* stats, float* norms, void* workspace, void* stream) {
  if (grads == nullptr || desc == nullptr) return AR_EINVAL;
  ar_status s = count_ok(n);
  if (s != AR_OK) return s;
  if (desc->kind != AR_NORM_L2 && desc->kind != AR_NORM_MAX) return AR_EINVAL;
  if (!(desc->max_norm > 0.0) || !(desc->eps >= 0.0) || !std::isfinite(desc->eps) || !std::isfinite(desc->grad_scale))
    return AR_EINVAL;
  if (!aligned(stats, 4) || !aligned(workspace, 16) || (norms != nullptr && !aligned(norms, 4))) return AR_EINVAL;
  if (!valid(grads, n) || (outs != nullptr && !valid(outs, n))) return AR_EINVAL;
  std::vector<GradTensor> t(n);
  Ranges ranges(size_t(2 * n + 3));
  for (int i = 0; i < n; ++i) {
    const ar_tensor& in = grads[i];
    const ar_tensor& out = outs != nullptr ? outs[i] : in;
    if (out.count != in.count || out.dtype != in.dtype) return AR_EINVAL;
    t[i] = {static_cast<const char*>(in.data), static_cast<char*>(out.data), in.count, in.dtype == AR_BF16};
    if (!clip || out.data != in.data) ranges.add(range(in, false));
  }
  for (int i = 0; clip && i < n; ++i) ranges.add(range(outs != nullptr ? outs[i] : grads[i], true));
  ranges.add(range(stats, 16, true));
  ranges.add(range(norms, norms != nullptr ? 4 * int64_t(n) : 0, true));
  ranges.add(range(workspace, kGradWorkspace, true));
  if (!ranges.apart()) return AR_EINVAL;
  if ((s = device_ready()) != AR_OK) return s;
  GradJob job = {};
  job.kind = desc->kind;
  halves(desc->max_norm, job.max_norm, job.max_norm_low);
  halves(desc->eps, job.eps, job.eps_low);
  job.grad_scale = desc->grad_scale;
  job.stats = stats;
  job.norms = norms;
  job.groups = workspace;
  job.partials = static_cast<char*>(workspace) + kGradPartials;
  return from_cuda(launch_grad_norm(t.data(), n, clip, job, static_cast<cudaStream_t>(stream)));
}

// Elements between a multiple of 8 and the first one; 255 where the arrays do
// not agree (16-byte accesses need a multiple of 4 of fp32, of 8 of bf16).
struct Phase {
  int of8 = -1, of4 = -1;
  bool alike = true;
  void add(const void* p, bool bf16) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p) / (bf16 ? 2 : 4);
    if (bf16) {
      alike = alike && (of8 < 0 || of8 == int(at % 8));
      of8 = int(at % 8);
    }
    alike = alike && (of4 < 0 || of4 == int(at % 4));
    of4 = int(at % 4);
  }
  uint8_t value() const { return !alike ? 255 : uint8_t(of8 >= 0 ? of8 : of4); }
};

}  // namespace

extern "C" {

ar_status ar_grad_workspace(int n_tensors, size_t* bytes) {
  if (bytes == nullptr) return AR_EINVAL;
  const ar_status s = count_ok(n_tensors);
  if (s == AR_OK) *bytes = size_t(kGradWorkspace);
  return s;
}

ar_status ar_grad_norm(const ar_tensor* grads, int n_tensors, const ar_norm_desc* desc, float* stats, float* norms,
                       void* workspace, void* stream) try {
  return grad_norm(grads, n_tensors, nullptr, false, desc, stats, norms, workspace, stream);
} catch (const std::bad_alloc&) {
  return AR_ENOMEM;
}

ar_status ar_grad_clip(const ar_tensor* grads, int n_tensors, const ar_tensor* outs, const ar_norm_desc* desc,
                       float* stats, float* norms, void* workspace, void* stream) try {
  return grad_norm(grads, n_tensors, outs, true, desc, stats, norms, workspace, stream);
} catch (const std::bad_alloc&) {
  return AR_ENOMEM;
}

ar_status ar_adamw_step(const ar_adamw_desc* desc, int n_tensors, const ar_tensor* params, const ar_tensor* grads,
                        const ar_tensor* exp_avgs, const ar_tensor* exp_avg_sqs, const ar_tensor* masters,
                        const ar_tensor* params_out, const ar_tensor* exp_avgs_out, const ar_tensor* exp_avg_sqs_out,
                        const ar_tensor* masters_out, const float* clip, void* stream) try {
  if (desc == nullptr) return AR_EINVAL;
  ar_status s = count_ok(n_tensors);
  if (s != AR_OK) return s;
  if (!std::isfinite(desc->lr) || !std::isfinite(desc->weight_decay) || !(desc->eps >= 0.0) || !std::isfinite(desc->eps) ||
      !(desc->beta1 >= 0.0 && desc->beta1 < 1.0) || !(desc->beta2 >= 0.0 && desc->beta2 < 1.0) ||
      !std::isfinite(desc->grad_scale))
    return AR_EINVAL;
  if (desc->device_step == nullptr ? desc->step < 1 : !aligned(desc->device_step, 8)) return AR_EINVAL;
  if (desc->device_lr != nullptr && !aligned(desc->device_lr, 4)) return AR_EINVAL;
  if (clip != nullptr && !aligned(clip, 4)) return AR_EINVAL;
  if (masters == nullptr && masters_out != nullptr) return AR_EINVAL;
  if (params_out == nullptr) params_out = params;
  if (exp_avgs_out == nullptr) exp_avgs_out = exp_avgs;
  if (exp_avg_sqs_out == nullptr) exp_avg_sqs_out = exp_avg_sqs;
  if (masters_out == nullptr) masters_out = masters;
  const int n = n_tensors;
  for (const ar_tensor* list : {params, grads, exp_avgs, exp_avg_sqs, params_out, exp_avgs_out, exp_avg_sqs_out})
    if (!valid(list, n)) return AR_EINVAL;
  std::vector<AdamEntry> e(n);
  bool in_place = true;
  for (int i = 0; i < n; ++i) {
    const ar_tensor &p = params[i], &g = grads[i], &m = exp_avgs[i], &v = exp_avg_sqs[i], &po = params_out[i],
                    &mo = exp_avgs_out[i], &vo = exp_avg_sqs_out[i];
    for (const ar_tensor* t : {&g, &m, &v, &po, &mo, &vo})
      if (t->count != p.count) return AR_EINVAL;
    if (po.dtype != p.dtype) return AR_EINVAL;
    for (const ar_tensor* t : {&m, &v, &mo, &vo})
      if (t->dtype != AR_F32) return AR_EINVAL;
    const bool has_master = masters != nullptr && masters[i].data != nullptr && p.count > 0;
    if (masters != nullptr && (masters_out[i].data != nullptr) != (masters[i].data != nullptr)) return AR_EINVAL;
    if (has_master)
      for (const ar_tensor* t : {&masters[i], &masters_out[i]})
        if (!valid(*t) || t->count != p.count || t->dtype != AR_F32) return AR_EINVAL;
    const ar_tensor &w = has_master ? masters[i] : p, &wo = has_master ? masters_out[i] : po;
    e[i] = {g.data, w.data, static_cast<const float*>(m.data), static_cast<const float*>(v.data), wo.data,
            has_master ? po.data : nullptr, static_cast<float*>(mo.data), static_cast<float*>(vo.data), p.count, 0,
            uint8_t(g.dtype == AR_BF16), uint8_t(w.dtype == AR_BF16), uint8_t(p.dtype == AR_BF16), 0};
    Phase ph;
    ph.add(g.data, g.dtype == AR_BF16);
    for (const void* f : {static_cast<const void*>(m.data), static_cast<const void*>(v.data),
                          static_cast<const void*>(mo.data), static_cast<const void*>(vo.data)})
      ph.add(f, false);
    ph.add(w.data, w.dtype == AR_BF16);
    ph.add(wo.data, w.dtype == AR_BF16);
    if (has_master) ph.add(po.data, p.dtype == AR_BF16);
    e[i].phase = ph.value();
    if (m.data != mo.data || v.data != vo.data || w.data != wo.data || p.data != po.data) in_place = false;
  }
  Ranges ranges(size_t(9 * n + 2));
  for (int i = 0; i < n; ++i) ranges.add(range(grads[i], false));
  const auto list = [&](auto in, auto out, int64_t size) {  // of the entries' arrays
    for (int i = 0; i < n; ++i)
      if (in(i) != out(i)) ranges.add(range(in(i), e[i].count * size, false));
    for (int i = 0; i < n; ++i) ranges.add(range(out(i), e[i].count * size, true));
  };
  list([&](int i) { return e[i].m; }, [&](int i) { return e[i].m_out; }, 4);
  list([&](int i) { return e[i].v; }, [&](int i) { return e[i].v_out; }, 4);
  for (int i = 0; i < n; ++i)
    if (e[i].w != e[i].w_out) ranges.add(range(e[i].w, e[i].count * (e[i].w_bf16 ? 2 : 4), false));
  for (int i = 0; i < n; ++i) ranges.add(range(e[i].w_out, e[i].count * (e[i].w_bf16 ? 2 : 4), true));
  for (int i = 0; i < n; ++i)
    if (e[i].p_out != nullptr) ranges.add(range(e[i].p_out, e[i].count * (e[i].p_bf16 ? 2 : 4), true));
  if (clip != nullptr) ranges.add(range(clip, 16, false));
  if (desc->device_step != nullptr) ranges.add(range(desc->device_step, 8, false));
  if (desc->device_lr != nullptr) ranges.add(range(desc->device_lr, 4, false));
  if (!ranges.apart()) return AR_EINVAL;
  if ((s = device_ready()) != AR_OK) return s;
  AdamJob job = {};
  job.rates = {float(desc->beta1), float(desc->beta2), float(1.0 - desc->beta1), float(1.0 - desc->beta2), 0.0f, 0.0f,
               float(desc->eps), 0.0f};
  job.step = std::max<int64_t>(desc->step, 1);
  const double log1 = std::log(desc->beta1), log2 = std::log(desc->beta2);  // (-inf for a beta of 0)
  job.rates.rate = float(desc->lr / -std::expm1(double(job.step) * log1));
  job.rates.inv_root = float(1.0 / std::sqrt(-std::expm1(double(job.step) * log2)));
  job.rates.keep = float(1.0 - desc->lr * desc->weight_decay);
  job.device_step = desc->device_step;
  job.device_lr = desc->device_lr;
  job.lr = float(desc->lr);
  job.weight_decay = float(desc->weight_decay);
  halves(log1, job.log1, job.log1_low);
  halves(log2, job.log2, job.log2_low);
  job.clip = clip;
  job.grad_scale = desc->grad_scale;
  job.in_place = in_place;
  return from_cuda(launch_adamw(e.data(), n, job, static_cast<cudaStream_t>(stream)));
} catch (const std::bad_alloc&) {
  return AR_ENOMEM;
}

}  // extern "C"
