// xent.hip -- softmax cross entropy of a linear head over a large vocabulary,
// and its gradient, without keeping the logits, for gfx950.
//
//   z = x W^T   lse_n = log sum_v exp z_nv   loss_n = lse_n - z_n,target(n)
//   dz = (exp(z - lse) - onehot) * grad      dx = dz W      dW = dz^T x
//
// These are the two ends of a replayed step (AWS Machine Learning Blog,
// "Detecting and recovering from silent data corruption on Amazon SageMaker
// HyperPod", section "Check 2": a replay's row starts with the loss bits), and
// the gradient recomputes the logits, which is the case of AEGIS' recompute
// check (review page, section "core method", item 4) whose original is never
// in memory: both passes can fingerprint the logits while they are in
// registers.
//
// Forward: one launch of logit tiles, each leaving its columns' running maximum
// and sum of exponentials and the targets' logits it holds, one that merges a
// row's tiles into its loss, one for the total (one for both for few tokens).  The
// tiles are computed as z^T (vocabulary down, tokens across), which puts 32 logits
// of one token into each lane (256 x 256; 4 to 16 in the smaller tiles): a token's
// maximum and sum need two shuffles.
// Gradient: the vocabulary in pieces; per piece the logit tiles again, whose
// epilogue writes dz (16-bit), then the two products of dz in one launch.  dx
// is summed over pieces and splits in fp32 in a fixed order.  Bound by the
// matrix cores (2 N V d operations forward, 6 N V d for the gradient), for up to
// about 200 tokens by reading W (and, for the gradient, reading it again and
// writing dW).
#include <algorithm>

#include "xent_device.h"

namespace sdc {
namespace {

// ---- copies of operands ---------------------------------------------------------
// A wave copies part of a row; 4096 x 2048 takes 8.3 us (4 TB/s).
constexpr uint32_t kPackCols = 2048;  // of one wave: four loads of 16 bytes in flight

template <bool VEC>
__global__ void __launch_bounds__(kBlock) pack_kernel(const PackArgs a) {
  const uint32_t r = wave_item_index(), l = threadIdx.x & 63u;
  if (r >= a.R) return;
  const bool live = !a.mask || has_target(a.mask[r], a.vocab);
  const unsigned char* src = a.src + (uint64_t)r * a.stride;
  uint16_t* dst = a.dst + (uint64_t)r * a.c_pad;
  const uint32_t end = min(a.c_pad, (blockIdx.y + 1u) * kPackCols);
#pragma unroll 4
  for (uint32_t c = blockIdx.y * kPackCols + l * 8u; c < end; c += 512u) {
    u32x4 v = {0u, 0u, 0u, 0u};
    if (live) {
      if (VEC) {
        v = *reinterpret_cast<const u32x4*>(src + c * 2u);
      } else if (c + 8u <= a.C) {
        v = *reinterpret_cast<const u32x4_at2*>(src + c * 2u);
      } else {
        uint32_t e[8];
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k)
          e[k] = c + k < a.C ? *reinterpret_cast<const uint16_t*>(src + (c + k) * 2u) : 0u;
        v = u32x4{e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16};
      }
    }
    *reinterpret_cast<u32x4*>(dst + c) = v;
  }
}

}  // namespace

int32_t launch_pack(const PackArgs& a, hipStream_t s) {
  const bool vec = a.C % 8 == 0 && a.stride % 16 == 0 && reinterpret_cast<uintptr_t>(a.src) % 16 == 0;
  const dim3 grid((a.R + kWaves - 1) / kWaves, (a.c_pad + kPackCols - 1) / kPackCols);
  if (vec) hipLaunchKernelGGL(pack_kernel<true>, grid, dim3(kBlock), 0, s, a);
  else hipLaunchKernelGGL(pack_kernel<false>, grid, dim3(kBlock), 0, s, a);
  return launch_status();
}

namespace {

// ---- dx's sum ---------------------------------------------------------------------
// dx = grad * the splits' sum, in split order; 0 for rows without a target.
// Bound by latency, so the loads of 16 splits are in flight at a time: 256
// splits of 5 x 163 took 32 us one by one and take 5.6.
template <class T>
__global__ void __launch_bounds__(256) dx_finish_kernel(const float* __restrict__ part, uint32_t splits,
                                                        uint32_t N, uint32_t d,
                                                        const int64_t* __restrict__ target, uint64_t vocab,
                                                        const float* __restrict__ grad,
                                                        uint16_t* __restrict__ dx) {
  const uint32_t n = blockIdx.x;
  const bool live = has_target(target[n], vocab);
  const float g = *grad * (1.0f / T::kDzScale);
  const uint32_t c = blockIdx.y * 256u + threadIdx.x;
  if (c >= d) return;
  float s = 0.0f;
  if (live) {
    const float* p = part + (uint64_t)n * d + c;
    const uint64_t step = (uint64_t)N * d;
    uint32_t k = 0;
    for (; k + 16 <= splits; k += 16) {
      float v[16];
#pragma unroll
      for (uint32_t i = 0; i < 16; ++i) v[i] = p[(k + i) * step];
#pragma unroll
      for (uint32_t i = 0; i < 16; ++i) s += v[i];
    }
    for (; k < splits; ++k) s += p[k * step];
  }
  dx[(uint64_t)n * d + c] = (uint16_t)T::bits(live ? s * g : 0.0f);
}

// ---- row results -------------------------------------------------------------------
// What the row kernels need of the logit tiles and of a head.
struct RowArgs {
  const float2* part;  // [N][n_vt]
  const float* hit;    // the target's logit (rows with a target)
  uint32_t n_vt, N;
  const int64_t* target;
  uint64_t vocab;
  float *loss, *lse;
  float* total;
  uint64_t* count;
};

// Token n by one wave: merges its tiles' maxima m and sums s.  The loss is
// (m - z_target) + ln s, both at least 0 as s holds the maximum's 1: near zero it
// keeps the digits that lse - z_target would lose to lse's size.  Lane 0
// stores; every lane returns the loss.
__device__ __forceinline__ float token_loss(const RowArgs& a, uint32_t n) {
  const uint32_t l = threadIdx.x & 63u;
  const bool live = has_target(a.target[n], a.vocab);
  const float hit = live ? a.hit[n] : 0.0f;
  float m = -__builtin_inff(), s = 0.0f;
  for (uint32_t k = l; k < a.n_vt; k += 512) {  // eight loads in flight
    float2 p[8];
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i)
      p[i] = k + 64u * i < a.n_vt ? a.part[(uint64_t)n * a.n_vt + k + 64u * i] : float2{-__builtin_inff(), 0.0f};
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) {
      const float M = __builtin_fmaxf(m, p[i].x);
      s = s * rescale(m, M) + p[i].y * rescale(p[i].x, M);
      m = M;
    }
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    const float pm = __shfl_xor(m, off), ps = __shfl_xor(s, off), M = __builtin_fmaxf(m, pm);
    s = s * rescale(m, M) + ps * rescale(pm, M);
    m = M;
  }
  const float ln = kLn2 * __builtin_amdgcn_logf(s), loss = live ? (m - hit) + ln : 0.0f;
  if (l == 0) {
    a.lse[n] = m + ln;
    a.loss[n] = loss;
  }
  return loss;
}

// One wave a token: bound by latency (4096 tokens with 197 tiles: 5.4 us).
__global__ void __launch_bounds__(kBlock) lse_kernel(const RowArgs a) {
  const uint32_t n = wave_item_index();
  if (n < a.N) token_loss(a, n);
}

// total = sum of the losses (in double, thread t adding t, t + 1024, ..., then
// a fixed tree; rounded once to fp32), count = rows with a target.
__device__ __forceinline__ void store_total(const RowArgs& a, const float* loss) {
  double s = 0.0;
  uint32_t c = 0;
  for (uint32_t k = threadIdx.x; k < a.N; k += 1024) {
    s += loss[k];
    c += has_target(a.target[k], a.vocab);
  }
  __shared__ double sw[16];
  __shared__ uint32_t cw[16];
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    s += __shfl_xor(s, off);
    c += __shfl_xor(c, off);
  }
  if ((threadIdx.x & 63) == 0) {
    sw[threadIdx.x >> 6] = s;
    cw[threadIdx.x >> 6] = c;
  }
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int i = 1; i < 16; ++i) {
    s += sw[i];
    c += cw[i];
  }
  *a.total = (float)s;
  if (a.count) *a.count = c;
}

// One workgroup, latency only (4096 losses: 4.8 us).
__global__ void __launch_bounds__(1024) loss_total_kernel(const RowArgs a) { store_total(a, a.loss); }

// Few tokens: their losses and the total in one launch of one workgroup (one
// token with 1002 tiles: 6.0 us; 19 with 387: 4.8).
constexpr uint32_t kFewTokens = 32;

__global__ void __launch_bounds__(1024) few_tokens_kernel(const RowArgs a) {
  __shared__ float losses[kFewTokens];
  for (uint32_t n = threadIdx.x >> 6; n < a.N; n += 16) {
    const float loss = token_loss(a, n);
    if ((threadIdx.x & 63u) == 0) losses[n] = loss;
  }
  __syncthreads();
  store_total(a, losses);
}

// The logits' row from its tiles' rows; with ref, a difference under col_mask
// adds 1 to *mismatch.
__global__ void __launch_bounds__(64) logit_row_kernel(const sdc_row* __restrict__ parts, uint32_t n,
                                                       const sdc_row* __restrict__ ref, uint32_t col_mask,
                                                       sdc_row* __restrict__ out,
                                                       uint32_t* __restrict__ mismatch) {
  Lane ln = merge_slots(parts, n, threadIdx.x);
  wave_reduce(ln);
  if (threadIdx.x != 0) return;
  const sdc_row r = {ln.s, ln.w, ln.x, ln.nf};
  if (ref) {
    const sdc_row o = *ref;
    const bool differs = ((col_mask & SDC_COL_SUM) && r.sum != o.sum) ||
                         ((col_mask & SDC_COL_WSUM) && r.wsum != o.wsum) ||
                         ((col_mask & SDC_COL_XOR) && r.xorsum != o.xorsum) ||
                         ((col_mask & SDC_COL_NONFINITE) && r.nonfinite != o.nonfinite);
    if (differs) atomicAdd(mismatch, 1u);
  }
  *out = r;
}

__global__ void __launch_bounds__(256) zero16_kernel(uint16_t* p, uint64_t n) {
  for (uint64_t i = blockIdx.x * 256ull + threadIdx.x; i < n; i += gridDim.x * 256ull) p[i] = 0;
}

}  // namespace

int32_t launch_merge_tile_rows(const sdc_row* parts, uint32_t n, const sdc_row* ref, uint32_t col_mask, sdc_row* row,
                               uint32_t* mismatch, hipStream_t s) {
  hipLaunchKernelGGL(logit_row_kernel, dim3(1), dim3(64), 0, s, parts, n, ref, col_mask, row, mismatch);
  return launch_status();
}

int32_t launch_zero16(uint16_t* p, uint64_t n, hipStream_t s) {
  hipLaunchKernelGGL(zero16_kernel, dim3(1024), dim3(256), 0, s, p, n);
  return launch_status();
}

// ---- host ----------------------------------------------------------------------------
uint32_t tiles(uint64_t n, uint32_t tile) { return (uint32_t)((n + tile - 1) / tile); }

// The tile of the logits' product, from the rounds that the CUs take: a tile has
// the work of its share of a 256 x 256 one at 1.15 times the cost for 128 x 128
// (twice the operand bytes per operation) and 2 for 64 x 64.  Larger tiles win
// where they fill whole rounds, smaller ones where they would leave CUs idle (a
// CU takes about 27 GB/s from beyond its L2 whatever is in flight) or tiles half
// empty.  Measured (loss, us, 64 / 128 / 256): 755 x 5296 x 688 49 / 76 / 132, 100 x
// 2048 x 8000 25 / 31 / 54, 500 x 2048 x 10000 46 / 38 / 56, 100 x 2048 x 50304 50 /
// 40 / 60, 300 x 1000 x 16000 32 / 27 / 35, 800 x 2048 x 50304 248 / 183 / 211, 2000 x
// 512 x 8000 37 / 30 / 26, 1500 x 4096 x 30000 646 / 352 / 303, 1000 x 1024 x 12000
// 45 / 38 / 37 (takes 128), 64 x 2048 x 50304 42 / 40 / 59 (takes 64).
// Up to 32 tokens fit a tile of 32, whose few accumulators leave the registers
// to keep several steps of loads in flight.  Measured against 64 x 64 and 128 x
// 128 (us): 5 x 8190 x 128255 379 / 417 / 450, 32 x 1001 x 20001 21 / 25 / 33, 32 x
// 2048 x 50304 42 / 42 / 41.
uint32_t logit_tile(uint64_t n, uint64_t vocab) {
  if (n <= kFew) return kFew;
  const auto cost = [&](uint32_t t, double each) {
    return (double)(((uint64_t)tiles(n, t) * tiles(vocab, t) + kCus - 1) / kCus) * each;
  };
  const double c256 = cost(256, 1.0), c128 = cost(128, 1.15 / 4), c64 = cost(64, 2.0 / 16);
  if (c64 < c128 && c64 < c256) return 64;
  return c128 < c256 ? 128 : 256;
}

// Vocabulary rows of a tile of 32 tokens: 128, or 64 where those would leave CUs
// idle.  Measured (loss, us, 64 / 128): 4 x 3312 x 8340 29 / 38, 10 x 4096 x
// 24000 40 / 47, 10 x 4096 x 32768 48 / 46, 19 x 836 x 49450 28 / 26.
uint32_t few_rows(uint64_t vocab) { return tiles(vocab, FewTile::M) < kCus ? FewTinyTile::M : FewTile::M; }

namespace {

constexpr uint64_t kPieceBytes = 256ull << 20;  // of the gradient's workspace that grows with the piece

struct Head {
  uint32_t N, d, V, d_pad;
  uint32_t tile, vtile;  // tokens (256, 128, 64 or kFew) and vocabulary rows of the logits' tiles
  uint32_t nt, vt;       // tiles of the tokens, of the whole vocabulary
  uint32_t ptile;        // 256 or 128, of the gradient's products
  bool copy_x, copy_w;   // the operand needs an aligned copy
  bool any;              // w's rows are read where they lie, off 16-byte boundaries
  uint32_t piece;        // vocabulary rows of a piece
  uint32_t pieces;
  uint32_t splits;       // of dx's sum over a piece
  uint32_t n_tiles;      // logit tiles over the whole vocabulary, piece by piece
};

int32_t check_head(const sdc_head* h) {
  if (h == nullptr) return SDC_ERR_INVALID;
  if (h->dtype != SDC_BF16 && h->dtype != SDC_F16) return SDC_ERR_DTYPE;
  if (h->d == 0 || h->vocab == 0 || h->flags != 0) return SDC_ERR_INVALID;
  if (h->n > 0 && (h->x == nullptr || h->target == nullptr)) return SDC_ERR_INVALID;
  if (h->w == nullptr || h->x_stride < h->d || h->w_stride < h->d) return SDC_ERR_INVALID;
  if (reinterpret_cast<uintptr_t>(h->x) % 2 || reinterpret_cast<uintptr_t>(h->w) % 2 ||
      reinterpret_cast<uintptr_t>(h->target) % 8)
    return SDC_ERR_ALIGN;
  if (h->n >= 1ull << 24 || h->d >= 1ull << 20 || h->vocab >= 1ull << 24 || h->x_stride >= 1ull << 40 ||
      h->w_stride >= 1ull << 40 || (uint64_t)tiles(h->n, 256) * (tiles(h->vocab, 256) + 4096) >= 1ull << 31)
    return SDC_ERR_RANGE;
  return SDC_OK;
}

// Parts that dx's sum over `rows` vocabulary rows is split into: a tile for each CU.
uint32_t dx_splits(uint64_t n, uint64_t d, uint64_t rows, uint32_t tile) {
  const uint32_t per = tiles(n, tile) * tiles(d, tile);
  return std::max(1u, std::min(kCus / std::max(per, 1u), tiles(rows, 256)));
}

// The tile of the gradient's two products over `rows` vocabulary rows: the
// time of all tiles, in k steps and the steps' worth of an epilogue (6 of a
// 256 x 256 tile, 3 of the smaller), over the workgroups that run at a time (one of
// 256, or two of 128 a CU, whose steps take 0.575 of the time), or that of the
// longest tile.  Measured (the whole gradient in us, 128 / 256): 4096 x 256 x
// 12800 145 / 193, 600 x 1024 x 20000 106 / 119, 256 x 4096 x 32000 312 / 317, 800 x
// 2048 x 50304 611 / 611, 2048 x 1024 x 16000 211 / 206, 1037 x 1000 x 32003 268 /
// 252, 1500 x 4096 x 30000 1185 / 1035.
uint32_t product_tile(uint64_t n, uint64_t d, uint64_t rows) {
  const auto steps = [&](uint32_t t) {
    const double k_dw = (double)tiles(n, kTileK), k_dx = (double)tiles(rows, kTileK);
    const double n_dw = (double)tiles(d, t) * tiles(rows, t), n_dx = (double)tiles(n, t) * tiles(d, t);
    const uint32_t splits = dx_splits(n, d, rows, t);
    const double all = n_dw * k_dw + n_dx * k_dx + (n_dw + n_dx * splits) * (t == 256 ? 6 : 3);
    return std::max(all / (t == 256 ? kCus : 2 * kCus), std::max(k_dw, k_dx / splits));
  };
  return 0.575 * steps(128) < steps(256) ? 128u : 256u;
}

// grad: the sizes of the gradient's pieces; else those of the forward pass,
// which needs pieces only for more than kLaunchTiles tiles (a copy of w, 16
// bytes for each of less than 2^24 rows, is below kPieceBytes).
Head plan_head(const sdc_head* h, bool grad) {
  Head p;
  p.N = (uint32_t)h->n;
  p.d = (uint32_t)h->d;
  p.V = (uint32_t)h->vocab;
  p.d_pad = (uint32_t)up(h->d, 8);
  // w is copied only where its rows are shorter than a load
  p.any = h->d % 8 || h->w_stride % 8 || reinterpret_cast<uintptr_t>(h->w) % 16;
  p.copy_w = p.any && h->d < 8;
  p.any = p.any && !p.copy_w;
  p.tile = logit_tile(p.N, p.V);
  p.vtile = p.tile == kFew ? few_rows(p.V) : p.tile;
  p.copy_x = (h->d % 8 || h->x_stride % 8 || reinterpret_cast<uintptr_t>(h->x) % 16) &&
             (p.tile != kFew || h->d < 8);  // few rows are read where they lie
  p.nt = tiles(p.N, p.tile);
  p.vt = tiles(p.V, p.vtile);
  // The most rows whose dz (and copy) take kPieceBytes; of the sizes from half
  // of that on, the one that needs the fewest rounds of a tile for each CU.
  const uint32_t nt = p.nt, vt = p.vt;
  const uint64_t col = (p.copy_w ? 2ull * p.d_pad : 0) + 2ull * p.N;
  uint32_t most = vt;
  if (grad && col * p.V > kPieceBytes) most = (uint32_t)std::max<uint64_t>(kPieceBytes / col / p.vtile, 1);
  most = std::min(most, std::max(kLaunchTiles / std::max(nt, 1u), 1u));
  uint32_t best = most;
  if (most < vt) {
    uint64_t least = ~0ull;
    for (uint32_t k = most; k >= (most + 1) / 2; --k) {
      const auto rounds_of = [&](uint64_t rows) { return (rows * nt + kCus - 1) / kCus; };
      const uint64_t rounds = (vt / k) * rounds_of(k) + rounds_of(vt % k);
      if (rounds < least) {
        least = rounds;
        best = k;
      }
    }
  }
  const uint64_t piece = (uint64_t)best * p.vtile;
  p.piece = (uint32_t)std::min<uint64_t>(piece, up(p.V, 8));
  p.pieces = (vt + best - 1) / best;
  p.ptile = product_tile(p.N, p.d, p.piece);
  p.splits = dx_splits(p.N, p.d, p.piece, p.ptile);
  p.n_tiles = nt * vt;
  return p;
}

struct Layout {
  uint64_t part, hit, rows, xc, wc, xm, dz, dxp, end;
};

Layout layout_head(const Head& p, bool grad) {
  Layout o;
  uint64_t at = 0;
  const auto take = [&](uint64_t bytes) {
    const uint64_t here = at;
    at = up(at + bytes, 256);
    return here;
  };
  o.rows = take(32ull * p.n_tiles);
  o.xc = take(p.copy_x ? 2ull * p.N * p.d_pad : 0);
  o.wc = take(p.copy_w ? 2ull * p.piece * p.d_pad : 0);
  o.part = o.hit = o.xm = o.dz = o.dxp = at;
  if (grad) {
    o.xm = take(2ull * p.N * p.d_pad);
    o.dz = take(2ull * p.N * p.piece);
    o.dxp = take(4ull * p.splits * p.N * p.d);
  } else {
    o.part = take(8ull * p.N * p.vt);
    o.hit = take(4ull * p.N);
  }
  o.end = std::max<uint64_t>(at, 256);
  return o;
}

// Operands of a piece, copied where they are not aligned.
int32_t piece_operands(const sdc_head* h, const Head& p, const Layout& o, unsigned char* ws, uint32_t v0,
                       uint32_t rows, LogitArgs* a, hipStream_t s) {
  const unsigned char* w = static_cast<const unsigned char*>(h->w) + 2ull * v0 * h->w_stride;
  int32_t st;
  a->x = Operand{static_cast<const unsigned char*>(h->x), 2 * h->x_stride, p.N, p.d};
  a->w = Operand{w, 2 * h->w_stride, rows, p.d};
  if (p.copy_x) {
    if (v0 == 0 && (st = launch_pack(PackArgs{a->x.p, a->x.stride, p.N, p.d, p.d_pad,
                                              reinterpret_cast<uint16_t*>(ws + o.xc), nullptr, 0}, s)))
      return st;
    a->x = Operand{ws + o.xc, 2ull * p.d_pad, p.N, p.d_pad};
  }
  if (p.copy_w) {
    if ((st = launch_pack(PackArgs{w, 2 * h->w_stride, rows, p.d, p.d_pad, reinterpret_cast<uint16_t*>(ws + o.wc),
                                   nullptr, 0}, s)))
      return st;
    a->w = Operand{ws + o.wc, 2ull * p.d_pad, rows, p.d_pad};
  }
  a->K = p.d;
  a->v0 = v0;
  a->nt = p.nt;
  a->n_tiles = tiles(rows, p.vtile) * a->nt;
  a->vocab = p.V;
  return SDC_OK;
}

int32_t merge_logit_row(const Layout& o, const Head& p, unsigned char* ws, const sdc_row* ref, uint32_t mask,
                        sdc_row* row, uint32_t* mismatch, hipStream_t s) {
  return launch_merge_tile_rows(reinterpret_cast<const sdc_row*>(ws + o.rows), p.n_tiles, ref, mask, row, mismatch, s);
}

}  // namespace
}  // namespace sdc

using namespace sdc;

extern "C" int32_t sdc_cross_entropy_ws_bytes(const sdc_head* h, uint64_t* h_bytes, uint64_t* h_grad_bytes) {
  int32_t st = check_head(h);
  if (st) return st;
  if (h_bytes) *h_bytes = layout_head(plan_head(h, false), false).end;
  if (h_grad_bytes) *h_grad_bytes = layout_head(plan_head(h, true), true).end;
  return SDC_OK;
}

extern "C" int32_t sdc_cross_entropy(const sdc_head* h, void* d_ws, uint64_t ws_bytes, float* d_loss,
                                     float* d_lse, float* d_total, uint64_t* d_count, sdc_row* d_row,
                                     sdc_stream_t stream) {
  int32_t st = check_head(h);
  if (st) return st;
  if (d_total == nullptr || d_ws == nullptr || (h->n > 0 && (d_loss == nullptr || d_lse == nullptr)))
    return SDC_ERR_INVALID;
  if (reinterpret_cast<uintptr_t>(d_ws) % 16 || reinterpret_cast<uintptr_t>(d_row) % 16 ||
      reinterpret_cast<uintptr_t>(d_loss) % 4 || reinterpret_cast<uintptr_t>(d_lse) % 4 ||
      reinterpret_cast<uintptr_t>(d_total) % 4 || reinterpret_cast<uintptr_t>(d_count) % 8)
    return SDC_ERR_ALIGN;
  const Head p = plan_head(h, false);
  const Layout o = layout_head(p, false);
  if (ws_bytes < o.end) return SDC_ERR_WORKSPACE;
  DeviceShape dev;
  if ((st = current_device_shape(&dev))) return st;
  hipStream_t s = as_stream(stream);
  unsigned char* ws = static_cast<unsigned char*>(d_ws);
  if (p.N > 0) {
    LogitArgs a = {};
    a.xcds = dev.xcds;
    a.target = h->target;
    a.part = reinterpret_cast<float2*>(ws + o.part);
    a.hit = reinterpret_cast<float*>(ws + o.hit);
    sdc_row* rows = reinterpret_cast<sdc_row*>(ws + o.rows);
    a.n_vt = p.vt;
    for (uint32_t k = 0; k < p.pieces; ++k) {
      const uint32_t v0 = k * p.piece, n = std::min(p.piece, p.V - v0);
      if ((st = piece_operands(h, p, o, ws, v0, n, &a, s))) return st;
      a.rows = d_row ? rows : nullptr;
      const HeadLaunch l = {h->dtype, p.vtile, p.ptile};
      if ((st = p.tile == kFew ? launch_logit_lse_few(l, a, s)
                : p.any        ? launch_logit_lse_any(l, a, s)
                               : launch_logit_lse16(l, a, s)))
        return st;
      rows += a.n_tiles;
      a.part += tiles(n, p.vtile);
    }
  }
  const RowArgs r = {reinterpret_cast<const float2*>(ws + o.part), reinterpret_cast<const float*>(ws + o.hit), p.vt,
                     p.N, h->target, h->vocab, d_loss, d_lse, d_total, d_count};
  if (p.N <= kFewTokens) {
    hipLaunchKernelGGL(few_tokens_kernel, dim3(1), dim3(1024), 0, s, r);
    st = launch_status();
  } else {
    hipLaunchKernelGGL(lse_kernel, dim3((p.N + kWaves - 1) / kWaves), dim3(kBlock), 0, s, r);
    if ((st = launch_status())) return st;
    hipLaunchKernelGGL(loss_total_kernel, dim3(1), dim3(1024), 0, s, r);
    st = launch_status();
  }
  if (st) return st;
  if (d_row) return merge_logit_row(o, p, ws, nullptr, 0, d_row, nullptr, s);
  return SDC_OK;
}

extern "C" int32_t sdc_cross_entropy_grad(const sdc_head* h, const float* d_lse, const float* d_grad, void* d_ws,
                                          uint64_t ws_bytes, void* d_dx, void* d_dw, const sdc_row* d_ref,
                                          uint32_t col_mask, sdc_row* d_row, uint32_t* d_mismatch,
                                          sdc_stream_t stream) {
  int32_t st = check_head(h);
  if (st) return st;
  if (d_grad == nullptr || d_ws == nullptr || (d_dx == nullptr && d_dw == nullptr) ||
      (h->n > 0 && d_lse == nullptr))
    return SDC_ERR_INVALID;
  if (d_ref != nullptr && (d_row == nullptr || d_mismatch == nullptr || col_mask == 0 || (col_mask & ~15u)))
    return SDC_ERR_INVALID;
  if (reinterpret_cast<uintptr_t>(d_ws) % 16 || reinterpret_cast<uintptr_t>(d_row) % 16 ||
      reinterpret_cast<uintptr_t>(d_ref) % 16 || reinterpret_cast<uintptr_t>(d_dx) % 2 ||
      reinterpret_cast<uintptr_t>(d_dw) % 2 || reinterpret_cast<uintptr_t>(d_lse) % 4 ||
      reinterpret_cast<uintptr_t>(d_grad) % 4 || reinterpret_cast<uintptr_t>(d_mismatch) % 4)
    return SDC_ERR_ALIGN;
  const Head p = plan_head(h, true);
  const Layout o = layout_head(p, true);
  if (ws_bytes < o.end) return SDC_ERR_WORKSPACE;
  DeviceShape dev;
  if ((st = current_device_shape(&dev))) return st;
  hipStream_t s = as_stream(stream);
  unsigned char* ws = static_cast<unsigned char*>(d_ws);
  if (p.N == 0) {
    if (d_dw && (st = launch_zero16(static_cast<uint16_t*>(d_dw), (uint64_t)p.V * p.d, s))) return st;
    return d_row ? merge_logit_row(o, p, ws, d_ref, col_mask, d_row, d_mismatch, s) : SDC_OK;
  }
  // x without what rows that have no target hold: dz is zero there, but 0 * NaN is not
  if (d_dw && (st = launch_pack(PackArgs{static_cast<const unsigned char*>(h->x), 2 * h->x_stride, p.N, p.d,
                                         p.d_pad, reinterpret_cast<uint16_t*>(ws + o.xm), h->target, h->vocab},
                                s)))
    return st;
  LogitArgs a = {};
  a.xcds = dev.xcds;
  a.target = h->target;
  a.lse = d_lse;
  a.dz = reinterpret_cast<uint16_t*>(ws + o.dz);
  sdc_row* rows = reinterpret_cast<sdc_row*>(ws + o.rows);
  float* dxp = reinterpret_cast<float*>(ws + o.dxp);
  for (uint32_t k = 0; k < p.pieces; ++k) {
    const uint32_t v0 = k * p.piece, n = std::min(p.piece, p.V - v0), v_pad = (uint32_t)up(n, 8);
    if ((st = piece_operands(h, p, o, ws, v0, n, &a, s))) return st;
    a.v_pad = v_pad;
    a.rows = d_row ? rows : nullptr;
    rows += a.n_tiles;
    ProductArgs x;
    x.w = a.w;
    x.dz = Operand{ws + o.dz, 2ull * v_pad, p.N, v_pad};
    x.x = Operand{ws + o.xm, 2ull * p.d_pad, p.N, p.d_pad};
    x.N = p.N;
    x.d = p.d;
    x.rows = n;
    x.xcds = dev.xcds;
    x.nt = tiles(p.N, p.ptile);
    x.md = tiles(p.d, p.ptile);
    x.n_dx = d_dx ? x.nt * x.md * p.splits : 0;
    x.n_dw = d_dw ? x.md * tiles(n, p.ptile) : 0;
    x.chunk = (uint32_t)up((n + p.splits - 1) / p.splits, kTileK);
    x.part = dxp;
    x.first = k == 0;
    x.grad = d_grad;
    x.dw = d_dw ? static_cast<uint16_t*>(d_dw) + (uint64_t)v0 * p.d : nullptr;
    const HeadLaunch l = {h->dtype, p.vtile, p.ptile};
    if ((st = p.tile == kFew ? launch_logit_dz_few(l, a, s)
              : p.any        ? launch_logit_dz_any(l, a, s)
                             : launch_logit_dz16(l, a, s)))
      return st;
    if ((st = p.any ? launch_products_any(l, x, s) : launch_products16(l, x, s))) return st;
  }
  if (d_dx) {
    st = for_dtype(h->dtype, [&](auto t) {
      typedef decltype(t) T;
      hipLaunchKernelGGL(dx_finish_kernel<T>, dim3(p.N, (p.d + 255) / 256), dim3(256), 0, s, dxp, p.splits, p.N, p.d,
                         h->target, h->vocab, d_grad, static_cast<uint16_t*>(d_dx));
      return launch_status();
    });
    if (st) return st;
  }
  if (d_row) return merge_logit_row(o, p, ws, d_ref, col_mask, d_row, d_mismatch, s);
  return SDC_OK;
}
