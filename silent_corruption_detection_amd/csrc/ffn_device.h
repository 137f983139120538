// ffn_device.h -- the tiled kernels of the gated feed-forward block (csrc/ffn.hip
// says what they compute), instantiated for weights whose rows lie at 16-byte
// boundaries (csrc/ffn16.hip), for any others (csrc/ffn_any.hip) and for few
// rows of x (csrc/ffn_few.hip).
#pragma once

#include "tile_device.h"

namespace sdc {

struct FfnArgs {
  Paired w;                // [f][d] each
  Operand x;               // rows of tokens
  uint32_t K, f, act;
  uint32_t nt, n_tiles, xcds;
  // forward
  uint16_t* h;             // [n][f]
  // gradient
  const uint16_t* dh;
  uint64_t dh_stride;      // elements
  uint16_t* dz;            // [n][2][f_pad]: dg, du
  uint32_t f_pad;
  // fingerprint of the projections: one partial row per tile, or null
  sdc_row* rows;
};

// All products of a gradient in one launch: dx's tiles first (their sums are the
// longer ones), then those of both weights.
struct FfnProductArgs {
  Operand wg, wu;          // [f][d]
  Operand dg, du;          // [N][f_pad]
  Operand x;               // [N][d]
  uint32_t N, d, f, xcds;
  uint32_t nt, md, mf;     // tiles of the tokens, of d, of f
  uint32_t n_dx, n_dw;     // tiles; n_dw: of both weights
  uint32_t chunk;          // k of a split of dx, over the gate's f (in whole steps) and then the up's
  float* part;             // [splits][N][d], or null: dx is stored by its one split
  uint16_t *dx, *dw_gate, *dw_up;
};

// tile: the rows of the two weights together of the projections' tile.
struct FfnLaunch {
  uint32_t dtype, tile;
};
int32_t launch_ffn16(const FfnLaunch& l, const FfnArgs& a, hipStream_t s);
int32_t launch_ffn_any(const FfnLaunch& l, const FfnArgs& a, hipStream_t s);
int32_t launch_ffn_few(const FfnLaunch& l, const FfnArgs& a, hipStream_t s);
int32_t launch_ffn_products16(const FfnLaunch& l, const FfnProductArgs& a, hipStream_t s);
int32_t launch_ffn_products_any(const FfnLaunch& l, const FfnProductArgs& a, hipStream_t s);

namespace {

// For few tokens with rows to spare: two groups a wave, one of each weight.
typedef Shape<64, 32, 2, 2, 4> FewPairTile;

// a = g y, the activation, and slope, its derivative, with y = 1 / (1 + exp(-t)):
//   silu       t = g                          slope = y + g y (1 - y)
//   gelu_tanh  t = 2 c (g + 0.044715 g^3)     slope = y + g y (1 - y) t'(g),   c = sqrt(2 / pi)
// (0.5 (1 + tanh(t / 2)) is y.)  Where y (1 - y) is 0, so is the second term, whatever
// its other factors overflow to.
__device__ __forceinline__ void activation(uint32_t act, float g, float* a, float* slope) {
  constexpr float c2 = 1.59576912160573071f, cubic = 0.044715f;
  float t = g, dt = 1.0f;
  if (act == SDC_ACT_GELU_TANH) {
    const float q = cubic * g * g;
    t = c2 * (g + q * g);
    dt = c2 * (1.0f + 3.0f * q);
  }
  const float e = __builtin_amdgcn_exp2f(-kLog2e * t);
  const float y = __builtin_amdgcn_rcpf(1.0f + e);
  const float bend = y * (1.0f - y);
  *a = g * y;
  *slope = bend == 0.0f ? y : y + g * bend * dt;
}

// The tile's part of the fingerprint row of the fp32 projections [n][2][f].
template <class S>
__device__ __forceinline__ void projections_row(const f32x4 (&acc)[S::I][S::J], const FfnArgs& a, uint32_t f0,
                                                uint32_t n0, sdc_row* out) {
  const Place<S> at;
  Lane ln;
#pragma unroll
  for (int j = 0; j < S::J; ++j) {
    const uint32_t n = n0 + at.col(j);
    if (n >= a.x.rows) continue;
#pragma unroll
    for (int up = 0; up < 2; ++up) {
      uint64_t s = 0, ws = 0;
#pragma unroll
      for (int i = up; i < S::I; i += 2)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if (f0 + i / 2 * 16 + r >= a.f) continue;
          const uint32_t x = __float_as_uint(acc[i][j][r]);
          s += x;
          ws += (uint64_t)(i / 2 * 16 + r) * x;
          ln.x ^= x;
          ln.nf += ((x & 0x7F800000u) + 0x00800000u) >> 31;
        }
      ln.s += s;
      ln.w += ws + (((uint64_t)n * 2u + up) * a.f + f0 + 1u) * s;
    }
  }
  store_tile_row<S::kThreads / 64>(ln, out);
}

// A tile of both projections (GRAD: computed again) and what is made of it.
// The rows of the two weights alternate by 16 (Paired), so a lane holds g and u of the
// same element in neighbouring accumulators, and both come from one pass over x.
//   forward  h = act(g) u, rounded once.
//   GRAD     dg = dh u act'(g), du = dh act(g), rounded to the inputs' type: the products
//            of the gradient take them as 16-bit operands, where the halves of a step
//            (2^-9 of a value in bf16, 2^-12 in fp16) average out over their sums.
// What is stored passes through LDS, so that it goes out (and dh comes in) in whole
// rows of the tile.  Bound by the matrix cores: 4096 x 2048 x 8192 takes 229 us (1200 TFLOP/s), and
// computed again for dg and du 277 us (992 TFLOP/s: dh is read, two results are stored); few tokens
// by reading the weights (1 x 8192 x 28672: 163 us, 5.8 TB/s).
template <class T, class S, RowsAt AT, bool ROW, bool GRAD>
__global__ void __launch_bounds__(S::kThreads) ffn_kernel(const FfnArgs a) {
  extern __shared__ __align__(16) unsigned char lds[];
  static_assert(S::I % 2 == 0, "a wave has whole pairs");
  constexpr uint32_t F = S::M / 2;  // of f in the tile
  const uint32_t id = xcd_run(blockIdx.x, a.n_tiles, a.xcds);
  const uint32_t f_at = id / a.nt * F, n0 = (id % a.nt) * S::N;
  const Place<S> at;
  f32x4 acc[S::I][S::J];
  gemm_tile<T, S, AT, false, false>(a.w, a.x, 2 * f_at, n0, 0, a.K, lds, acc);
  const uint32_t local = at.wm * (F / S::WM) + (at.lane >> 4) * 4u;  // the lane's first element of f in the tile
  if constexpr (ROW) projections_row<S>(acc, a, f_at + local, n0, a.rows + id);
  uint16_t* st = reinterpret_cast<uint16_t*>(lds);  // [token][gate's F, up's F]
  const uint32_t t = threadIdx.x, ch = t % (F / 8) * 8u, k0 = t / (F / 8);
  constexpr uint32_t kStep = S::kThreads / (F / 8);
  if constexpr (GRAD) {
    for (uint32_t k = k0; k < S::N; k += kStep) {
      const uint32_t n = n0 + k, c = f_at + ch;
      u32x4 v = {0u, 0u, 0u, 0u};
      if (n < a.x.rows && c < a.f) {
        const uint16_t* p = a.dh + (uint64_t)n * a.dh_stride + c;
        if (c + 8u <= a.f) {
          v = *reinterpret_cast<const u32x4_at2*>(p);
        } else {
          uint32_t e[8];
#pragma unroll
          for (uint32_t i = 0; i < 8; ++i) e[i] = c + i < a.f ? p[i] : 0u;
          v = u32x4{e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16};
        }
      }
      *reinterpret_cast<u32x4*>(st + k * stage_row<S>() + ch) = v;
    }
    __syncthreads();
  }
#pragma unroll
  for (int j = 0; j < S::J; ++j)
#pragma unroll
    for (int i = 0; i < S::I; i += 2) {
      uint16_t* p = st + at.col(j) * stage_row<S>() + local + i / 2 * 16;
      uint32_t b[4], c[4];
      if constexpr (GRAD) {
        const uint2 dh = *reinterpret_cast<const uint2*>(p);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float y, slope;
          activation(a.act, acc[i][j][r], &y, &slope);
          const float d = T::value((r < 2 ? dh.x : dh.y) >> (16 * (r & 1)) & 0xFFFFu);
          const bool in = f_at + local + i / 2 * 16 + r < a.f;  // the padding is 0, whatever 0 times u is
          b[r] = T::bits(in ? d * acc[i + 1][j][r] * slope : 0.0f);
          c[r] = T::bits(in ? d * y : 0.0f);
        }
        *reinterpret_cast<uint2*>(p + F) = uint2{c[0] | c[1] << 16, c[2] | c[3] << 16};
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float y, slope;
          activation(a.act, acc[i][j][r], &y, &slope);
          b[r] = T::bits(y * acc[i + 1][j][r]);
        }
      }
      *reinterpret_cast<uint2*>(p) = uint2{b[0] | b[1] << 16, b[2] | b[3] << 16};
    }
  __syncthreads();
#pragma unroll 4
  for (uint32_t k = k0; k < S::N; k += kStep) {
    const uint32_t n = n0 + k, c = f_at + ch;
    if (n >= a.x.rows) continue;
    const uint16_t* s = st + k * stage_row<S>() + ch;
    if constexpr (GRAD) {
      if (c < a.f_pad) {
        uint16_t* p = a.dz + (uint64_t)n * 2u * a.f_pad + c;
        *reinterpret_cast<u32x4*>(p) = *reinterpret_cast<const u32x4*>(s);
        *reinterpret_cast<u32x4*>(p + a.f_pad) = *reinterpret_cast<const u32x4*>(s + F);
      }
    } else if (c < a.f) {
      store8(a.h + (uint64_t)n * a.f + c, s, a.f - c);
    }
  }
}

// A tile of C^T (M down, N across) to 16-bit rows of `width` elements, through LDS.
template <class T, class S>
__device__ __forceinline__ void store_tile(const f32x4 (&acc)[S::I][S::J], uint16_t* out, uint32_t m0, uint32_t n0,
                                           uint32_t width, uint32_t rows, unsigned char* lds) {
  const Place<S> at;
  uint16_t* st = reinterpret_cast<uint16_t*>(lds);
#pragma unroll
  for (int j = 0; j < S::J; ++j)
#pragma unroll
    for (int i = 0; i < S::I; ++i) {
      uint32_t b[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) b[r] = T::bits(acc[i][j][r]);
      *reinterpret_cast<uint2*>(st + at.col(j) * stage_row<S>() + at.row(i)) =
          uint2{b[0] | b[1] << 16, b[2] | b[3] << 16};
    }
  __syncthreads();
  const uint32_t t = threadIdx.x, ch = t % (S::M / 8) * 8u;
#pragma unroll 4
  for (uint32_t k = t / (S::M / 8); k < S::N; k += S::kThreads / (S::M / 8)) {
    const uint32_t n = n0 + k, m = m0 + ch;
    if (n < rows && m < width) store8(out + (uint64_t)n * width + m, st + k * stage_row<S>() + ch, width - m);
  }
}

// dx^T = Wg^T dg^T + Wu^T du^T, over a split of the two sums' k.
template <class T, class S, RowsAt AT>
__device__ __forceinline__ void ffn_dx_tile(const FfnProductArgs& a, uint32_t id, unsigned char* lds) {
  const uint32_t n0 = (id % a.nt) * S::N, rest = id / a.nt;
  const uint32_t m0 = (rest % a.md) * S::M, split = rest / a.md;
  const uint32_t whole = (a.f + kTileK - 1) / kTileK * kTileK;
  const uint32_t k0 = min(split * a.chunk, 2u * whole), k1 = min(k0 + a.chunk, 2u * whole);
  f32x4 acc[S::I][S::J];
#pragma unroll
  for (int i = 0; i < S::I; ++i)
#pragma unroll
    for (int j = 0; j < S::J; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  if (k0 < min(k1, whole)) gemm_tile<T, S, AT, true, false, true>(a.wg, a.dg, m0, n0, k0, min(k1, whole), lds, acc);
  if (max(k0, whole) < k1)
    gemm_tile<T, S, AT, true, false, true>(a.wu, a.du, m0, n0, max(k0, whole) - whole, k1 - whole, lds, acc);
  if (!a.part) return store_tile<T, S>(acc, a.dx, m0, n0, a.d, a.N, lds);
  const Place<S> at;
  float* out = a.part + (uint64_t)split * a.N * a.d;
#pragma unroll
  for (int j = 0; j < S::J; ++j) {
    const uint32_t n = n0 + at.col(j);
    if (n >= a.N) continue;
#pragma unroll
    for (int i = 0; i < S::I; ++i) {
      const uint32_t m = m0 + at.row(i);
      float* p = out + (uint64_t)n * a.d + m;
      if (a.d % 4 == 0) {
        if (m < a.d) *reinterpret_cast<f32x4*>(p) = acc[i][j];
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (m + r < a.d) p[r] = acc[i][j][r];
      }
    }
  }
}

template <class T, class S>
__device__ __forceinline__ void ffn_dw_tile(const FfnProductArgs& a, uint32_t id, unsigned char* lds) {
  const bool up = id >= a.n_dw / 2;
  if (up) id -= a.n_dw / 2;
  const uint32_t m0 = (id % a.md) * S::M, n0 = (id / a.md) * S::N;
  f32x4 acc[S::I][S::J];
  gemm_tile<T, S, kAt16, true, true>(a.x, up ? a.du : a.dg, m0, n0, 0, a.N, lds, acc);
  store_tile<T, S>(acc, up ? a.dw_up : a.dw_gate, m0, n0, a.d, a.f, lds);
}

// dx and both weights' gradients (see FfnProductArgs).  Bound by the matrix cores: 4096 x 2048 x
// 8192 takes 433 us (1270 TFLOP/s), 2048 x 8192 x 28672 3450 us (1115 TFLOP/s).
template <class T, class S, RowsAt AT>
__global__ void __launch_bounds__(S::kThreads) ffn_products_kernel(const FfnProductArgs a) {
  extern __shared__ __align__(16) unsigned char lds[];
  if (blockIdx.x < a.n_dx) ffn_dx_tile<T, S, AT>(a, xcd_run(blockIdx.x, a.n_dx, a.xcds), lds);
  else ffn_dw_tile<T, S>(a, xcd_run(blockIdx.x - a.n_dx, a.n_dw, a.xcds), lds);
}

template <RowsAt AT>
int32_t launch_ffn(const FfnLaunch& l, const FfnArgs& a, hipStream_t s) {
  return for_dtype(l.dtype, [&](auto type) {
    typedef decltype(type) T;
    const auto launch = [&](auto shape) {
      typedef decltype(shape) S;
      const dim3 grid(a.n_tiles), block(S::kThreads);
      constexpr uint32_t bytes = lds_bytes<S>();
      if (a.dz && a.rows) hipLaunchKernelGGL((ffn_kernel<T, S, AT, true, true>), grid, block, bytes, s, a);
      else if (a.dz) hipLaunchKernelGGL((ffn_kernel<T, S, AT, false, true>), grid, block, bytes, s, a);
      else if (a.rows) hipLaunchKernelGGL((ffn_kernel<T, S, AT, true, false>), grid, block, bytes, s, a);
      else hipLaunchKernelGGL((ffn_kernel<T, S, AT, false, false>), grid, block, bytes, s, a);
      return launch_status();
    };
    if constexpr (AT == kDeep) return l.tile == 128 ? launch(FewTile()) : launch(FewPairTile());
    else return l.tile == 256 ? launch(BigTile()) : l.tile == 128 ? launch(SmallTile()) : launch(TinyTile());
  });
}

template <RowsAt AT>
int32_t launch_ffn_products(const FfnLaunch& l, const FfnProductArgs& a, hipStream_t s) {
  return for_dtype(l.dtype, [&](auto type) {
    typedef decltype(type) T;
    const auto launch = [&](auto shape) {
      typedef decltype(shape) S;
      hipLaunchKernelGGL((ffn_products_kernel<T, S, AT>), dim3(a.n_dx + a.n_dw), dim3(S::kThreads), lds_bytes<S>(), s,
                         a);
      return launch_status();
    };
    return l.tile == 256 ? launch(BigTile()) : launch(SmallTile());
  });
}

}  // namespace
}  // namespace sdc
