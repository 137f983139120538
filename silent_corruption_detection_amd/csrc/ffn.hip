// ffn.hip -- the gated feed-forward block's first half and its gradient, for gfx950.
//
//   g = x Wg^T   u = x Wu^T   h = act(g) u
//   dg = dh u act'(g)   du = dh act(g)
//   dx = dg Wg + du Wu   dWg = dg^T x   dWu = du^T x
//
// The gradient computes g and u again, which is the recomputation of AEGIS' check
// (review page, section "core method", item 4) whose original is never in memory:
// both passes can fingerprint the projections while they are in registers.
//
// Forward: one launch of matrix-product tiles, whose rows alternate between the two
// weights, with the activation and the product in the epilogue.  Gradient: the same
// tiles, whose epilogue writes dg and du (16 bits), then all three products in one
// launch; dx is summed over both weights in one tile, in fp32, in a fixed order.
// Bound by the matrix cores (4 N d f operations forward, 12 N d f for the gradient),
// for up to about 200 tokens by reading the weights (and, for the gradient, reading them
// again and writing theirs).
#include <cmath>

#include "ffn_device.h"

namespace sdc {
namespace {

// dx = the splits' sum, in split order.
template <class T>
__global__ void __launch_bounds__(256) ffn_dx_finish_kernel(const float* __restrict__ part, uint32_t splits,
                                                            uint64_t n, uint16_t* __restrict__ dx) {
  for (uint64_t i = blockIdx.x * 256ull + threadIdx.x; i < n; i += gridDim.x * 256ull) {
    float s = 0.0f;
    uint32_t k = 0;
    for (; k + 8 <= splits; k += 8) {  // eight loads in flight
      float v[8];
#pragma unroll
      for (uint32_t j = 0; j < 8; ++j) v[j] = part[(k + j) * n + i];
#pragma unroll
      for (uint32_t j = 0; j < 8; ++j) s += v[j];
    }
    for (; k < splits; ++k) s += part[k * n + i];
    dx[i] = (uint16_t)T::bits(s);
  }
}

// ---- host ----------------------------------------------------------------------------
struct Ffn {
  uint32_t N, d, f, d_pad, f_pad;
  uint32_t tile, rows;         // tokens of the projections' tiles, rows of both weights together
  uint32_t nt, n_tiles;
  bool copy_x, copy_w, any;    // copies for operands that need them; weights read off 16-byte boundaries
  uint32_t ptile, splits, chunk;
};

bool unaligned(const void* p, uint64_t stride, uint64_t d) {
  return d % 8 || stride % 8 || reinterpret_cast<uintptr_t>(p) % 16;
}

int32_t check_ffn(const sdc_ffn* b) {
  if (b == nullptr) return SDC_ERR_INVALID;
  if (b->dtype != SDC_BF16 && b->dtype != SDC_F16) return SDC_ERR_DTYPE;
  if (b->d == 0 || b->f == 0 || (b->act != SDC_ACT_SILU && b->act != SDC_ACT_GELU_TANH)) return SDC_ERR_INVALID;
  if (b->n > 0 && b->x == nullptr) return SDC_ERR_INVALID;
  if (b->w_gate == nullptr || b->w_up == nullptr || b->x_stride < b->d || b->w_gate_stride < b->d ||
      b->w_up_stride < b->d)
    return SDC_ERR_INVALID;
  if (reinterpret_cast<uintptr_t>(b->x) % 2 || reinterpret_cast<uintptr_t>(b->w_gate) % 2 ||
      reinterpret_cast<uintptr_t>(b->w_up) % 2)
    return SDC_ERR_ALIGN;
  if (b->n >= 1ull << 24 || b->d >= 1ull << 20 || b->f >= 1ull << 23 || b->x_stride >= 1ull << 40 ||
      b->w_gate_stride >= 1ull << 40 || b->w_up_stride >= 1ull << 40)
    return SDC_ERR_RANGE;
  // launches of the largest and the smallest tiles (those that are chosen for few)
  const uint64_t n = tiles(b->n, 128), d = tiles(b->d, 128), f = tiles(2 * b->f, 128);
  if (n * f >= kLaunchTiles || n * d >= kLaunchTiles / 2 || d * f >= kLaunchTiles / 2) return SDC_ERR_RANGE;
  return SDC_OK;
}

// The tile of the gradient's products and the splits of dx's sum.  A tile takes a step
// for each 64 of its k and some for its epilogue (6 steps of a 256 x 256 tile, 3 of a 128 x
// 128 one, whose steps take 0.575 of the time with two workgroups a CU); dx's are the
// longest, and are split as far as one of them would outlast the whole work's share of
// a CU.  Measured (bf16, us of the whole gradient with 256 / 128): 256 x 1024 x 4096 39.8 /
// 35.3, 1037 x 1000 x 2731 65.2 / 70.7, 1024 x 2048 x 8192 195 / 211, 4096 x 2048 x 8192 702 /
// 819; the rule takes the faster each time.
void plan_products(Ffn* p) {
  const double steps_f = tiles(p->f, kTileK), steps_n = tiles(p->N, kTileK);
  double best = 0.0;
  for (const uint32_t t : {256u, 128u}) {
    const double epilogue = t == 256 ? 6 : 3, slots = t == 256 ? kCus : 2 * kCus;
    const double n_dx = (double)tiles(p->N, t) * tiles(p->d, t), n_dw = 2.0 * tiles(p->d, t) * tiles(p->f, t);
    const double share = (n_dx * (2 * steps_f + epilogue) + n_dw * (steps_n + epilogue)) / slots;
    const double most = std::min<double>(2 * steps_f, 64);
    const double splits = std::min(most, std::max(1.0, std::ceil(2 * steps_f / std::max(share, 8.0))));
    const double time = std::max(share, 2 * steps_f / splits) * (t == 256 ? 1.0 : 0.575);
    if (t == 256 || time < best) {
      best = time;
      p->ptile = t;
      p->splits = (uint32_t)splits;
    }
  }
  p->chunk = (uint32_t)up((2 * (uint64_t)steps_f * kTileK + p->splits - 1) / p->splits, kTileK);
}

Ffn plan_ffn(const sdc_ffn* b) {
  Ffn p;
  p.N = (uint32_t)b->n;
  p.d = (uint32_t)b->d;
  p.f = (uint32_t)b->f;
  p.d_pad = (uint32_t)up(p.d, 8);
  p.f_pad = (uint32_t)up(p.f, 8);
  p.any = unaligned(b->w_gate, b->w_gate_stride, b->d) || unaligned(b->w_up, b->w_up_stride, b->d);
  p.copy_w = p.any && b->d < 8;  // rows shorter than a load
  p.any = p.any && !p.copy_w;
  p.tile = logit_tile(p.N, 2 * p.f);
  p.rows = p.tile == kFew ? few_rows(2 * p.f) : p.tile;
  p.copy_x = unaligned(b->x, b->x_stride, b->d) && (p.tile != kFew || b->d < 8);  // few rows are read where they lie
  p.nt = tiles(p.N, p.tile);
  p.n_tiles = p.nt * tiles(p.f, p.rows / 2);
  plan_products(&p);
  return p;
}

struct FfnLayout {
  uint64_t rows, xc, wc, dz, part, end;
};

FfnLayout layout_ffn(const sdc_ffn* b, const Ffn& p, bool grad) {
  FfnLayout o;
  uint64_t at = 0;
  const auto take = [&](uint64_t bytes) {
    const uint64_t here = at;
    at = up(at + bytes, 256);
    return here;
  };
  o.rows = take(32ull * p.n_tiles);
  // the gradient's product over the tokens takes x at 16-byte boundaries whatever the tiles do
  o.xc = take(p.copy_x || (grad && unaligned(b->x, b->x_stride, b->d)) ? 2ull * p.N * p.d_pad : 0);
  o.wc = take(p.copy_w ? 4ull * p.f * p.d_pad : 0);
  o.dz = take(grad ? 4ull * p.N * p.f_pad : 0);
  o.part = take(grad && p.splits > 1 ? 4ull * p.splits * p.N * p.d : 0);
  o.end = std::max<uint64_t>(at, 256);
  return o;
}

// Operands, copied where they have to be (x also where the gradient's product needs it).
int32_t ffn_operands(const sdc_ffn* b, const Ffn& p, const FfnLayout& o, unsigned char* ws, bool grad, FfnArgs* a,
                     Operand* x, hipStream_t s) {
  int32_t st;
  const Operand in = {static_cast<const unsigned char*>(b->x), 2 * b->x_stride, p.N, p.d};
  *x = in;
  if (p.copy_x || (grad && unaligned(b->x, b->x_stride, b->d))) {
    if ((st = launch_pack(PackArgs{in.p, in.stride, p.N, p.d, p.d_pad, reinterpret_cast<uint16_t*>(ws + o.xc), nullptr,
                                   0}, s)))
      return st;
    *x = Operand{ws + o.xc, 2ull * p.d_pad, p.N, p.d_pad};
  }
  a->x = p.copy_x ? *x : in;
  a->w.a = Operand{static_cast<const unsigned char*>(b->w_gate), 2 * b->w_gate_stride, p.f, p.d};
  a->w.b = Operand{static_cast<const unsigned char*>(b->w_up), 2 * b->w_up_stride, p.f, p.d};
  if (p.copy_w) {
    unsigned char* to = ws + o.wc;
    for (Operand* w : {&a->w.a, &a->w.b}) {
      if ((st = launch_pack(PackArgs{w->p, w->stride, p.f, p.d, p.d_pad, reinterpret_cast<uint16_t*>(to), nullptr, 0},
                            s)))
        return st;
      *w = Operand{to, 2ull * p.d_pad, p.f, p.d_pad};
      to += 2ull * p.f * p.d_pad;
    }
  }
  a->K = p.d;
  a->f = p.f;
  a->act = b->act;
  a->nt = p.nt;
  a->n_tiles = p.n_tiles;
  return SDC_OK;
}

int32_t launch_projections(const sdc_ffn* b, const Ffn& p, const FfnArgs& a, hipStream_t s) {
  const FfnLaunch l = {b->dtype, p.rows};
  return p.tile == kFew ? launch_ffn_few(l, a, s) : p.any ? launch_ffn_any(l, a, s) : launch_ffn16(l, a, s);
}

}  // namespace
}  // namespace sdc

using namespace sdc;

extern "C" int32_t sdc_gated_ffn_ws_bytes(const sdc_ffn* h, uint64_t* h_bytes, uint64_t* h_grad_bytes) {
  int32_t st = check_ffn(h);
  if (st) return st;
  const Ffn p = plan_ffn(h);
  if (h_bytes) *h_bytes = layout_ffn(h, p, false).end;
  if (h_grad_bytes) *h_grad_bytes = layout_ffn(h, p, true).end;
  return SDC_OK;
}

extern "C" int32_t sdc_gated_ffn(const sdc_ffn* b, void* d_ws, uint64_t ws_bytes, void* d_h, sdc_row* d_row,
                                 sdc_stream_t stream) {
  int32_t st = check_ffn(b);
  if (st) return st;
  if (d_ws == nullptr || (b->n > 0 && d_h == nullptr)) return SDC_ERR_INVALID;
  if (reinterpret_cast<uintptr_t>(d_ws) % 16 || reinterpret_cast<uintptr_t>(d_row) % 16 ||
      reinterpret_cast<uintptr_t>(d_h) % 2)
    return SDC_ERR_ALIGN;
  const Ffn p = plan_ffn(b);
  const FfnLayout o = layout_ffn(b, p, false);
  if (ws_bytes < o.end) return SDC_ERR_WORKSPACE;
  DeviceShape dev;
  if ((st = current_device_shape(&dev))) return st;
  hipStream_t s = as_stream(stream);
  unsigned char* ws = static_cast<unsigned char*>(d_ws);
  if (p.N > 0) {
    FfnArgs a = {};
    Operand x;
    if ((st = ffn_operands(b, p, o, ws, false, &a, &x, s))) return st;
    a.xcds = dev.xcds;
    a.h = static_cast<uint16_t*>(d_h);
    a.rows = d_row ? reinterpret_cast<sdc_row*>(ws + o.rows) : nullptr;
    if ((st = launch_projections(b, p, a, s))) return st;
  }
  if (d_row)
    return launch_merge_tile_rows(reinterpret_cast<const sdc_row*>(ws + o.rows), p.n_tiles, nullptr, 0, d_row, nullptr,
                                  s);
  return SDC_OK;
}

extern "C" int32_t sdc_gated_ffn_grad(const sdc_ffn* b, const void* d_dh, uint64_t dh_stride, void* d_ws,
                                      uint64_t ws_bytes, void* d_dx, void* d_dw_gate, void* d_dw_up,
                                      const sdc_row* d_ref, uint32_t col_mask, sdc_row* d_row, uint32_t* d_mismatch,
                                      sdc_stream_t stream) {
  int32_t st = check_ffn(b);
  if (st) return st;
  if (d_ws == nullptr || (b->n > 0 && d_dx == nullptr && d_dw_gate == nullptr) || (d_dw_gate == nullptr) != (d_dw_up == nullptr) ||
      (b->n > 0 && d_dh == nullptr) || dh_stride < b->f)
    return SDC_ERR_INVALID;
  if (d_ref != nullptr && (d_row == nullptr || d_mismatch == nullptr || col_mask == 0 || (col_mask & ~15u)))
    return SDC_ERR_INVALID;
  if (reinterpret_cast<uintptr_t>(d_ws) % 16 || reinterpret_cast<uintptr_t>(d_row) % 16 ||
      reinterpret_cast<uintptr_t>(d_ref) % 16 || reinterpret_cast<uintptr_t>(d_dh) % 2 ||
      reinterpret_cast<uintptr_t>(d_dx) % 2 || reinterpret_cast<uintptr_t>(d_dw_gate) % 2 ||
      reinterpret_cast<uintptr_t>(d_dw_up) % 2 || reinterpret_cast<uintptr_t>(d_mismatch) % 4)
    return SDC_ERR_ALIGN;
  if (dh_stride >= 1ull << 40) return SDC_ERR_RANGE;
  const Ffn p = plan_ffn(b);
  const FfnLayout o = layout_ffn(b, p, true);
  if (ws_bytes < o.end) return SDC_ERR_WORKSPACE;
  DeviceShape dev;
  if ((st = current_device_shape(&dev))) return st;
  hipStream_t s = as_stream(stream);
  unsigned char* ws = static_cast<unsigned char*>(d_ws);
  const sdc_row* rows = reinterpret_cast<const sdc_row*>(ws + o.rows);
  if (p.N == 0) {
    for (void* w : {d_dw_gate, d_dw_up})
      if (w && (st = launch_zero16(static_cast<uint16_t*>(w), (uint64_t)p.f * p.d, s))) return st;
    return d_row ? launch_merge_tile_rows(rows, 0, d_ref, col_mask, d_row, d_mismatch, s) : SDC_OK;
  }
  FfnArgs a = {};
  FfnProductArgs x = {};
  if ((st = ffn_operands(b, p, o, ws, true, &a, &x.x, s))) return st;
  a.xcds = dev.xcds;
  a.dh = static_cast<const uint16_t*>(d_dh);
  a.dh_stride = dh_stride;
  a.dz = reinterpret_cast<uint16_t*>(ws + o.dz);
  a.f_pad = p.f_pad;
  a.rows = d_row ? reinterpret_cast<sdc_row*>(ws + o.rows) : nullptr;
  if ((st = launch_projections(b, p, a, s))) return st;
  x.wg = a.w.a;
  x.wu = a.w.b;
  x.dg = Operand{ws + o.dz, 4ull * p.f_pad, p.N, p.f_pad};
  x.du = Operand{ws + o.dz + 2ull * p.f_pad, 4ull * p.f_pad, p.N, p.f_pad};
  x.N = p.N;
  x.d = p.d;
  x.f = p.f;
  x.xcds = dev.xcds;
  x.nt = tiles(p.N, p.ptile);
  x.md = tiles(p.d, p.ptile);
  x.mf = tiles(p.f, p.ptile);
  x.n_dx = d_dx ? x.nt * x.md * p.splits : 0;
  x.n_dw = d_dw_gate ? 2 * x.md * x.mf : 0;
  x.chunk = p.chunk;
  x.part = p.splits > 1 ? reinterpret_cast<float*>(ws + o.part) : nullptr;
  x.dx = static_cast<uint16_t*>(d_dx);
  x.dw_gate = static_cast<uint16_t*>(d_dw_gate);
  x.dw_up = static_cast<uint16_t*>(d_dw_up);
  const FfnLaunch l = {b->dtype, p.ptile};
  if ((st = p.any ? launch_ffn_products_any(l, x, s) : launch_ffn_products16(l, x, s))) return st;
  if (d_dx && x.part) {
    const uint64_t n = (uint64_t)p.N * p.d;
    const dim3 grid((uint32_t)std::min<uint64_t>((n + 255) / 256, 1u << 16));
    st = for_dtype(b->dtype, [&](auto t) {
      hipLaunchKernelGGL(ffn_dx_finish_kernel<decltype(t)>, grid, dim3(256), 0, s, x.part, p.splits, n, x.dx);
      return launch_status();
    });
    if (st) return st;
  }
  return d_row ? launch_merge_tile_rows(rows, p.n_tiles, d_ref, col_mask, d_row, d_mismatch, s) : SDC_OK;
}
