// adamw.hip -- the AdamW step over a tensor list for gfx950: the plan, the
// gate that decides on the device whether and how the step is taken, and the
// merge of the fingerprint rows.  The update kernels are in adamw_device.h.
//
// A step is one launch for the gate, one for each kernel class in the list
// (usually one or two), and, where rows are asked for, one merge.
#include <algorithm>
#include <cmath>
#include <vector>

#include "adamw_device.h"

namespace sdc {
namespace {

// beta1^t and beta2^t by squaring, in double (t in the thousands would lose
// digits in fp32): off by at most t 2^-53 of themselves, less than fp32 shows
// up to 2^28 steps.  The gate takes 2.2 us with this and
// 4.9 with pow where its inputs are in a cache.
__device__ __forceinline__ double2 powers(double b1, double b2, uint64_t t) {
  double2 r = {1.0, 1.0};
  for (; t; t >>= 1) {
    if (t & 1) {
      r.x *= b1;
      r.y *= b2;
    }
    b1 *= b1;
    b2 *= b2;
  }
  return r;
}

// The gate: skip, clip and bias corrections, one thread per parameter group,
// so nothing of a step waits for the host.
__global__ void __launch_bounds__(64) adamw_gate_kernel(sdc_adamw_control* control,
                                                        const sdc_adamw_group* __restrict__ groups,
                                                        uint32_t n_groups,
                                                        const double* __restrict__ sq_total,
                                                        const uint32_t* __restrict__ flag,
                                                        double max_norm, double grad_scale,
                                                        AdamwGate* __restrict__ gate,
                                                        AdamwCoef* __restrict__ coef) {
  const uint64_t done = control->step, seed = control->seed;
  const double total = sq_total ? *sq_total : 0.0;
  const bool skip = (flag && *flag != 0) || !__builtin_isfinite((float)total);
  const uint64_t t = done + (skip ? 0 : 1);
  sdc_adamw_group g = groups[min(threadIdx.x, n_groups - 1u)];
  __syncthreads();  // every thread has read the control block
  if (threadIdx.x == 0) {
    double scale = grad_scale;
    if (max_norm > 0.0) scale *= fmin(1.0, max_norm / (sqrt(total) * grad_scale + 1e-6));
    if (skip) control->skipped += 1;
    control->step = t;
    control->grad_scale = (float)scale;
    control->skip = skip;
    constexpr uint32_t kSeed = 0x9E3779B1u, kStep = 0x85157AF5u;
    *gate = AdamwGate{(float)scale, skip, (uint32_t)seed * kSeed + (uint32_t)t * kStep,
                      (uint32_t)(seed >> 32) * kSeed + (uint32_t)(t >> 32) * kStep + 0x6C8E9CF5u};
  }
  for (uint32_t k = threadIdx.x; k < n_groups; k += 64) {
    if (k >= 64) g = groups[k];
    const double2 p = powers(g.beta1, g.beta2, t);
    // an eps below fp32's normal numbers has no fp32 reciprocal: m = v = 0 would give 0 Inf
    const float eps = (float)g.eps < 0x1p-126f ? 0x1p-126f : (float)g.eps;
    coef[k] = AdamwCoef{(float)g.beta1, (float)(1.0 - g.beta1), (float)g.beta2, (float)(1.0 - g.beta2),
                        (float)(g.lr / (1.0 - p.x)), (float)(1.0 / sqrt(1.0 - p.y)), eps,
                        (float)(1.0 - g.lr * g.weight_decay)};
  }
}

// Rows of the tensors of several items (or of none), one wave each, or one
// workgroup.
template <bool WIDE>
__global__ void __launch_bounds__(kBlock) adamw_merge_kernel(const PlanSplit* __restrict__ split,
                                                             uint32_t n_split,
                                                             const sdc_row* __restrict__ partials,
                                                             sdc_row* __restrict__ rows) {
  const uint32_t e = WIDE ? blockIdx.x : wave_item_index();
  if (e >= n_split) return;
  const PlanSplit sp = split[e];
  const uint32_t l = WIDE ? threadIdx.x : threadIdx.x & 63u;
  Lane ln = merge_slots<WIDE ? kBlock : 64>(partials + sp.first, sp.count, l);
  if constexpr (WIDE) block_reduce(ln);
  else wave_reduce(ln);
  if (l == 0) store_row(rows + sp.row, ln, ln.w);
}

// A grid has fewer than 2^32 threads: a launch takes at most this many items of
// each kind, and the merge one wave for each tensor.
constexpr uint64_t kLaunchItems = 1ull << 23, kMaxTensors = 1ull << 25;

struct Layout {
  uint64_t n_items = 0, n_split = 0, n_slots = 0, total_elems = 0;
  uint64_t n_block[kAdamwClasses] = {}, n_wave[kAdamwClasses] = {};
  AdamwOffsets off{};
};

bool float_dtype(uint32_t d) { return d == SDC_F32 || d == SDC_BF16 || d == SDC_F16; }

bool aligned(const void* p, uint32_t es) { return reinterpret_cast<uintptr_t>(p) % es == 0; }

int32_t check_tensor(const sdc_adamw_tensor& t, uint32_t n_groups) {
  if (!float_dtype(t.param_dtype) || !float_dtype(t.grad_dtype)) return SDC_ERR_DTYPE;
  if (t.state_dtype != SDC_F32 && t.state_dtype != SDC_FP8_E4M3) return SDC_ERR_DTYPE;
  if (t.group >= n_groups) return SDC_ERR_INVALID;
  if (t.numel >= 1ull << 48) return SDC_ERR_RANGE;
  if (t.numel == 0) return SDC_OK;
  const bool eight = t.state_dtype == SDC_FP8_E4M3;
  if (!t.param || !t.exp_avg || !t.exp_avg_sq) return SDC_ERR_INVALID;
  if (eight != (t.exp_avg_scale != nullptr) || eight != (t.exp_avg_sq_scale != nullptr))
    return SDC_ERR_INVALID;
  if (t.master && t.param_dtype == SDC_F32) return SDC_ERR_INVALID;
  if (!aligned(t.param, element_size(t.param_dtype)) || !aligned(t.grad, element_size(t.grad_dtype)) ||
      !aligned(t.master, 4) || !aligned(t.exp_avg, eight ? 1 : 4) || !aligned(t.exp_avg_sq, eight ? 1 : 4))
    return SDC_ERR_ALIGN;
  return SDC_OK;
}

uint32_t class_of(const sdc_adamw_tensor& t) {
  const uint32_t p = t.param_dtype == SDC_F32 ? 0u : t.master ? 2u : 1u;
  const uint32_t g = (t.grad_dtype == SDC_F32 || !t.grad) ? 0u : 1u;
  return adamw_class(p, g, t.state_dtype == SDC_FP8_E4M3);
}

// Elements of a tensor with fp32 states past the 16-byte boundary at or below
// its exp_avg: its first item is that much shorter, so that the others start
// on a boundary.
uint64_t shift_of(const sdc_adamw_tensor& t) {
  return t.state_dtype == SDC_FP8_E4M3 ? 0 : (reinterpret_cast<uintptr_t>(t.exp_avg) >> 2) & 3;
}

uint64_t items_of(const sdc_adamw_tensor& t) {
  return t.numel ? (t.numel + shift_of(t) + kAdamwItemElems - 1) / kAdamwItemElems : 0;
}

bool of_wave(const sdc_adamw_tensor& t) { return t.numel + shift_of(t) <= kAdamwWaveElems; }

int32_t layout_adamw(const sdc_adamw_tensor* t, uint64_t n, uint32_t n_groups, Layout* L) {
  if ((n > 0 && t == nullptr) || n_groups == 0 || n_groups > 65536) return SDC_ERR_INVALID;
  if (n >= kMaxTensors) return SDC_ERR_RANGE;
  for (uint64_t k = 0; k < n; ++k) {
    if (int32_t st = check_tensor(t[k], n_groups)) return st;
    L->total_elems += t[k].numel;
    if (L->total_elems >= 1ull << 48) return SDC_ERR_RANGE;
    const uint64_t items = items_of(t[k]);
    L->n_items += items;
    if (L->n_items > kMaxGrid) return SDC_ERR_RANGE;
    if (items != 1) {
      L->n_split += 1;
      L->n_slots += items;
    }
    if (items == 0) continue;
    const uint32_t c = class_of(t[k]);
    if (of_wave(t[k])) L->n_wave[c] += 1;
    else L->n_block[c] += items;
  }
  L->off = adamw_offsets(n, n_groups, L->n_items, L->n_split, L->n_slots);
  return SDC_OK;
}

// Bytes of memory from start to end that a step reads or writes.
struct MemSpan {
  uint64_t start, end : 63, written : 1;
  bool operator<(const MemSpan& o) const { return start < o.start; }
};

// Whether something that a step writes overlaps another tensor of the list: the
// spans in order of their starts, against the furthest end of those before.  A
// column of pointers is usually in order by itself, so columns are merged.
bool overlapping(const sdc_adamw_tensor* t, uint64_t n) {
  std::vector<MemSpan> spans;
  const auto column = [&](auto&& place) {
    const size_t first = spans.size();
    for (uint64_t k = 0; k < n; ++k) {
      const MemSpan s = place(t[k]);
      if (t[k].numel && s.start) spans.push_back(s);
    }
    const auto mid = spans.begin() + (ptrdiff_t)first;
    if (!std::is_sorted(mid, spans.end())) std::sort(mid, spans.end());
    std::inplace_merge(spans.begin(), mid, spans.end());
  };
  const auto span = [](const void* p, uint64_t bytes, bool written) {
    const uint64_t a = reinterpret_cast<uintptr_t>(p);
    return MemSpan{a, a + bytes, written};
  };
  typedef const sdc_adamw_tensor& Tensor;
  // tensors without a gradient: their weights are read, for their rows
  const auto state = [&](Tensor x, const void* p) {
    return span(x.grad ? p : nullptr, x.numel * (x.state_dtype == SDC_F32 ? 4 : 1), true);
  };
  const auto scale = [&](Tensor x, const void* p) {
    return span(x.grad ? p : nullptr, (x.numel + kStateBlock - 1) / kStateBlock, true);
  };
  column([&](Tensor x) { return span(x.param, x.numel * element_size(x.param_dtype), x.grad != nullptr); });
  column([&](Tensor x) { return span(x.grad, x.numel * element_size(x.grad_dtype), false); });
  column([&](Tensor x) { return state(x, x.exp_avg); });
  column([&](Tensor x) { return state(x, x.exp_avg_sq); });
  column([&](Tensor x) { return span(x.grad ? x.master : nullptr, x.numel * 4, true); });
  column([&](Tensor x) { return scale(x, x.exp_avg_scale); });
  column([&](Tensor x) { return scale(x, x.exp_avg_sq_scale); });
  uint64_t read = 0, written = 0;  // furthest ends
  for (const MemSpan& s : spans) {
    if (s.start < written || (s.written && s.start < read)) return true;
    uint64_t& end = s.written ? written : read;
    end = std::max<uint64_t>(end, s.end);
  }
  return false;
}

void pack_adamw(const sdc_adamw_tensor* t, uint64_t n, const Layout& L, std::vector<unsigned char>& img) {
  img.assign(L.off.partials, 0);
  AdamwDesc* desc = reinterpret_cast<AdamwDesc*>(img.data() + L.off.desc);
  AdamwItem* items = reinterpret_cast<AdamwItem*>(img.data() + L.off.items);
  PlanSplit* split = reinterpret_cast<PlanSplit*>(img.data() + L.off.split);
  uint64_t block[kAdamwClasses], wave[kAdamwClasses], at = 0, first = 0, slot = 0, ns = 0;
  for (uint32_t c = 0; c < kAdamwClasses; ++c) {
    block[c] = at;
    wave[c] = at + L.n_block[c];
    at += L.n_block[c] + L.n_wave[c];
  }
  for (uint64_t k = 0; k < n; ++k) {
    const sdc_adamw_tensor& x = t[k];
    desc[k] = AdamwDesc{x.param, x.grad, x.exp_avg, x.exp_avg_sq, x.master, x.exp_avg_scale,
                        x.exp_avg_sq_scale, first, x.group, x.param_dtype, x.grad_dtype, 0};
    first += x.numel;
    const uint64_t count = items_of(x);
    if (count != 1) split[ns++] = PlanSplit{(uint32_t)k, (uint32_t)slot, (uint32_t)count, 0};
    if (count == 0) continue;
    const uint32_t c = class_of(x);
    uint64_t& next = of_wave(x) ? wave[c] : block[c];
    for (uint64_t s = 0, len = kAdamwItemElems - shift_of(x); s < x.numel; s += len, len = kAdamwItemElems) {
      const uint64_t left = x.numel - s;
      items[next++] = AdamwItem{s, (uint32_t)std::min(len, left), (uint32_t)k, count == 1 ? 0u : (uint32_t)slot++,
                                count == 1, 0};
    }
  }
}

void fill_info(const Layout& L, uint64_t n, uint32_t n_groups, sdc_adamw_info* h) {
  h->magic = kAdamwMagic;
  h->n_tensors = n;
  h->n_groups = n_groups;
  h->n_items = L.n_items;
  h->n_split = L.n_split;
  h->n_slots = L.n_slots;
  h->total_elems = L.total_elems;
  h->plan_bytes = L.off.end;
  for (uint32_t c = 0; c < kAdamwClasses; ++c) {
    h->n_block[c] = L.n_block[c];
    h->n_wave[c] = L.n_wave[c];
  }
}

bool adamw_info_ok(const sdc_adamw_info* h) {
  if (h->magic != kAdamwMagic || h->n_items > kMaxGrid || h->n_split > h->n_tensors ||
      h->n_tensors >= kMaxTensors || h->n_groups == 0 || h->n_groups > 65536 || h->n_slots > h->n_items)
    return false;
  uint64_t items = 0;
  for (uint32_t c = 0; c < kAdamwClasses; ++c) {
    if (h->n_block[c] > kMaxGrid || h->n_wave[c] > kMaxGrid) return false;
    items += h->n_block[c] + h->n_wave[c];
  }
  return items == h->n_items &&
         h->plan_bytes >= adamw_offsets(h->n_tensors, h->n_groups, h->n_items, h->n_split, h->n_slots).end;
}

}  // namespace
}  // namespace sdc

using namespace sdc;

extern "C" int32_t sdc_adamw_plan_bytes(const sdc_adamw_tensor* h_tensors, uint64_t n, uint32_t n_groups,
                                        uint64_t* h_bytes) {
  if (h_bytes == nullptr) return SDC_ERR_INVALID;
  Layout L;
  if (int32_t st = layout_adamw(h_tensors, n, n_groups, &L)) return st;
  *h_bytes = L.off.end;
  return SDC_OK;
}

extern "C" int32_t sdc_adamw_plan_build(const sdc_adamw_tensor* h_tensors, uint64_t n, uint32_t n_groups,
                                        void* d_plan, uint64_t plan_bytes, sdc_adamw_info* h_info,
                                        sdc_stream_t stream) {
  if (d_plan == nullptr || h_info == nullptr) return SDC_ERR_INVALID;
  Layout L;
  int32_t st = layout_adamw(h_tensors, n, n_groups, &L);
  if (st) return st;
  std::vector<unsigned char> img;
  try {
    if (overlapping(h_tensors, n)) return SDC_ERR_INVALID;
    if (plan_bytes < L.off.end) return SDC_ERR_WORKSPACE;
    if (!aligned(d_plan, 16)) return SDC_ERR_ALIGN;
    pack_adamw(h_tensors, n, L, img);
  } catch (...) {
    return SDC_ERR_RANGE;  // host allocation failed
  }
  hipStream_t s = as_stream(stream);
  st = hip_status(hipMemcpyAsync(d_plan, img.data(), img.size(), hipMemcpyHostToDevice, s));
  if (st) return st;
  st = hip_status(hipStreamSynchronize(s));
  if (st) return st;
  fill_info(L, n, n_groups, h_info);
  return SDC_OK;
}

extern "C" int32_t sdc_adamw_step(void* d_plan, const sdc_adamw_info* h_info,
                                  const sdc_adamw_group* d_groups, sdc_adamw_control* d_control,
                                  const double* d_sq_total, const uint32_t* d_flag, double max_norm,
                                  double grad_scale, sdc_row* d_rows, sdc_stream_t stream) {
  if (d_plan == nullptr || h_info == nullptr || d_groups == nullptr || d_control == nullptr)
    return SDC_ERR_INVALID;
  if (!adamw_info_ok(h_info)) return SDC_ERR_PLAN;
  if (!(max_norm >= 0.0) || (max_norm > 0.0 && d_sq_total == nullptr) || !(grad_scale > 0.0) ||
      !std::isfinite(max_norm) || !std::isfinite(grad_scale))
    return SDC_ERR_INVALID;
  if (!aligned(d_groups, 8) || !aligned(d_control, 8) || !aligned(d_sq_total, 8) || !aligned(d_flag, 4) ||
      !aligned(d_rows, 16))
    return SDC_ERR_ALIGN;
  hipStream_t s = as_stream(stream);
  unsigned char* base = static_cast<unsigned char*>(d_plan);
  const AdamwOffsets o = adamw_offsets(h_info->n_tensors, h_info->n_groups, h_info->n_items,
                                       h_info->n_split, h_info->n_slots);
  AdamwGate* gate = reinterpret_cast<AdamwGate*>(base + o.gate);
  AdamwCoef* coef = reinterpret_cast<AdamwCoef*>(base + o.coef);
  hipLaunchKernelGGL(adamw_gate_kernel, dim3(1), dim3(64), 0, s, d_control, d_groups,
                     (uint32_t)h_info->n_groups, d_sq_total, d_flag, max_norm, grad_scale, gate, coef);
  int32_t st = launch_status();
  if (st) return st;
  AdamwArgs a{gate, coef, reinterpret_cast<const AdamwDesc*>(base + o.desc),
              reinterpret_cast<const AdamwItem*>(base + o.items), 0, 0,
              reinterpret_cast<sdc_row*>(base + o.partials), d_rows};
  for (uint32_t c = 0; c < kAdamwClasses; ++c) {
    for (uint64_t block = h_info->n_block[c], wave = h_info->n_wave[c]; block + wave > 0;) {
      a.n_block = (uint32_t)std::min(block, kLaunchItems);
      a.n_wave = block > kLaunchItems ? 0u : (uint32_t)std::min(wave, kLaunchItems);
      st = (c & 1) ? launch_adamw8(c, a, s) : launch_adamw32(c, a, s);
      if (st) return st;
      a.items += a.n_block + a.n_wave;
      block -= a.n_block;
      wave -= a.n_wave;
    }
  }
  if (d_rows && h_info->n_split) {
    // A workgroup a tensor where the average has more rows than a wave has in
    // flight at a time (18 tensors of 0.96B weights, the longest of 50,304 rows:
    // 21 us; a wave each 71).
    const bool wide = h_info->n_slots / h_info->n_split >= 64 * kMergeUnroll;
    const dim3 grid((uint32_t)(wide ? h_info->n_split : (h_info->n_split + kWaves - 1) / kWaves));
    const PlanSplit* split = reinterpret_cast<const PlanSplit*>(base + o.split);
    const uint32_t n = (uint32_t)h_info->n_split;
    if (wide) hipLaunchKernelGGL(adamw_merge_kernel<true>, grid, dim3(kBlock), 0, s, split, n, a.partials, d_rows);
    else hipLaunchKernelGGL(adamw_merge_kernel<false>, grid, dim3(kBlock), 0, s, split, n, a.partials, d_rows);
    return launch_status();
  }
  return SDC_OK;
}
