// xent_device.h -- the tiled kernels of the cross-entropy head (csrc/xent.hip
// says what they compute), instantiated for weights whose rows lie at 16-byte
// boundaries (csrc/xent16.hip), for any others (csrc/xent_any.hip) and for
// few rows of x (csrc/xent_few.hip).
#pragma once

#include <algorithm>
#include <type_traits>

#include "fingerprint_device.h"
#include "gemm_device.h"

namespace sdc {

struct LogitArgs {
  Operand w, x;            // rows of the vocabulary (from v0 on), rows of tokens
  uint32_t K;              // elements of a row
  uint32_t v0;             // vocabulary index of w's first row
  uint32_t nt;             // token tiles
  uint32_t n_tiles, xcds;
  uint64_t vocab;
  const int64_t* target;
  // forward: [token][tile] maxima and sums, and the target's logit of each token
  float2* part;
  uint32_t n_vt;
  float* hit;
  // gradient
  const float* lse;
  uint16_t* dz;            // [x.rows][v_pad]
  uint32_t v_pad;
  // fingerprint of the logits: one partial row per tile, or null
  sdc_row* rows;
};

// Both products of a piece in one launch: dx's tiles first (they are the
// longer ones), then dW's, so that the chip fills up once.
struct ProductArgs {
  Operand w, dz, x;    // [piece rows][d], [N][v_pad], [N][d] with the rows without a target zero
  uint32_t N, d, rows, xcds;
  uint32_t nt, md;     // token tiles, tiles of d
  uint32_t n_dx, n_dw; // tiles
  uint32_t chunk;      // k of a split of dx
  float* part;         // [splits][N][d]
  uint32_t first;      // 1: the first piece stores, later ones add
  const float* grad;
  uint16_t* dw;        // of the piece's first row
};

// Launches over the tiles of one piece; tile: the rows of W of the logits'
// product's (256, 128 or 64), ptile: 256 or 128, of the gradient's.
struct HeadLaunch {
  uint32_t dtype, tile, ptile;
};
int32_t launch_logit_lse16(const HeadLaunch& h, const LogitArgs& a, hipStream_t s);
int32_t launch_logit_lse_any(const HeadLaunch& h, const LogitArgs& a, hipStream_t s);
int32_t launch_logit_lse_few(const HeadLaunch& h, const LogitArgs& a, hipStream_t s);
int32_t launch_logit_dz16(const HeadLaunch& h, const LogitArgs& a, hipStream_t s);
int32_t launch_logit_dz_any(const HeadLaunch& h, const LogitArgs& a, hipStream_t s);
int32_t launch_logit_dz_few(const HeadLaunch& h, const LogitArgs& a, hipStream_t s);
int32_t launch_products16(const HeadLaunch& h, const ProductArgs& x, hipStream_t s);
int32_t launch_products_any(const HeadLaunch& h, const ProductArgs& x, hipStream_t s);

namespace {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.693147180559945309417f;
// 16-bit elements of a staged row of M, padded off the banks
template <class S>
constexpr uint32_t stage_row() { return S::M + 8; }
template <class S>
constexpr uint32_t lds_bytes() { return std::max(S::kLds, S::N * stage_row<S>() * 2); }
static_assert(lds_bytes<BigTile>() + 1024 <= 160u * 1024u, "one workgroup fits a CU");

typedef uint32_t u32x4_at2 __attribute__((ext_vector_type(4), aligned(2)));

__device__ __forceinline__ bool has_target(int64_t t, uint64_t vocab) { return (uint64_t)t < vocab; }

// exp(x).  What it is called for is a difference of logits, taken before the
// factor log2(e): x log2(e) - M log2(e) would hold the rounding of M log2(e),
// which is no longer small beside the difference from |M| of 1e5 on and passes
// any exponent from 3e9 on.
__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

// exp(m - M) of a running maximum m <= M, also where both are the same infinity
__device__ __forceinline__ float rescale(float m, float M) {
  return m == M ? 1.0f : exp_of(m - M);
}

// ---- logit tiles ------------------------------------------------------------------

// The target of the token of a lane's column j, counted from the lane's first row
// of the tile (at.row(0), vocabulary row `first`): logit (i, r) is the target's
// where this is 16 i + r.  kNoTarget: none.  At most 2^24 rows, so a difference,
// also a negative one, is never kNoTarget.
constexpr uint32_t kNoTarget = 0x80000000u;
template <class S>
__device__ __forceinline__ uint32_t target_from(const LogitArgs& a, uint32_t n, uint32_t first) {
  const int64_t t = a.target[min(n, a.x.rows - 1u)];
  return has_target(t, a.vocab) && n < a.x.rows ? (uint32_t)t - first : kNoTarget;
}

// The tile's part of the fingerprint row of the fp32 logits [N][V].
template <class S>
__device__ __forceinline__ void tile_row(const f32x4 (&acc)[S::I][S::J], const LogitArgs& a, uint32_t m0,
                                         uint32_t n0, sdc_row* out) {
  const Place<S> at;
  Lane ln;
#pragma unroll
  for (int j = 0; j < S::J; ++j) {
    const uint32_t n = n0 + at.col(j);
    if (n >= a.x.rows) continue;
    uint64_t s = 0, ws = 0;
#pragma unroll
    for (int i = 0; i < S::I; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (m0 + at.row(i) + r >= a.w.rows) continue;
        const uint32_t x = __float_as_uint(acc[i][j][r]);
        s += x;
        ws += (uint64_t)(i * 16 + r) * x;
        ln.x ^= x;
        ln.nf += ((x & 0x7F800000u) + 0x00800000u) >> 31;
      }
    ln.s += s;
    ln.w += ws + ((uint64_t)n * a.vocab + a.v0 + m0 + at.row(0) + 1u) * s;
  }
  wave_reduce(ln);
  constexpr int kW = S::kThreads / 64;
  __shared__ uint64_t waves[4][kW];
  const uint32_t wave = threadIdx.x >> 6;
  if (at.lane == 0) {
    waves[0][wave] = ln.s;
    waves[1][wave] = ln.w;
    waves[2][wave] = ln.x;
    waves[3][wave] = ln.nf;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 1; i < kW; ++i) {
      ln.s += waves[0][i];
      ln.w += waves[1][i];
      ln.x ^= waves[2][i];
      ln.nf += waves[3][i];
    }
    ulonglong2* d = reinterpret_cast<ulonglong2*>(out);
    d[0] = ulonglong2{ln.s, ln.w};
    d[1] = ulonglong2{ln.x, ln.nf};
  }
}

// Maximum m and sum of exp(z - m) of each token over the tile's vocabulary rows:
// in a lane over its logits of the token, over the four lanes of its column by
// two shuffles, over the waves through LDS.  The lane that has the target's logit
// stores it, so that the loss is made of the logits whose sum (and fingerprint)
// was taken: a product of its own, summed in another order, would differ in the
// last bits, and could exceed the largest logit.  Bound by the matrix cores; 4096 x
// 50304 x 2048 takes 828 us of a trace on average (1020 TFLOP/s; 876 with the row).
template <class T, class S, RowsAt AT, bool ROW>
__global__ void __launch_bounds__(S::kThreads) logit_lse_kernel(const LogitArgs a) {
  extern __shared__ __align__(16) unsigned char lds[];
  const uint32_t id = xcd_run(blockIdx.x, a.n_tiles, a.xcds), vt = id / a.nt;
  const uint32_t m0 = vt * S::M, n0 = (id % a.nt) * S::N;
  const Place<S> at;
  uint32_t hit[S::J];  // read during the product
#pragma unroll
  for (int j = 0; j < S::J; ++j) hit[j] = target_from<S>(a, n0 + at.col(j), a.v0 + m0 + at.row(0));
  f32x4 acc[S::I][S::J];
  gemm_tile<T, S, AT, false, false>(a.w, a.x, m0, n0, 0, a.K, lds, acc);
  float2* half = reinterpret_cast<float2*>(lds);  // [wm][token of the tile]
#pragma unroll
  for (int j = 0; j < S::J; ++j) {
    float m = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < S::I; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (m0 + at.row(i) + r < a.w.rows) m = __builtin_fmaxf(m, acc[i][j][r]);
    m = __builtin_fmaxf(m, __shfl_xor(m, 16));
    m = __builtin_fmaxf(m, __shfl_xor(m, 32));
    const float shift = __builtin_isinf(m) ? 0.0f : m;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < S::I; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (m0 + at.row(i) + r < a.w.rows)
          s += exp_of(acc[i][j][r] - shift);
    s += __shfl_xor(s, 16);
    s += __shfl_xor(s, 32);
    if (at.lane < 16) half[at.wm * S::N + at.col(j)] = float2{m, s};
    if (hit[j] < S::I * 16u && (hit[j] & 15u) < 4u && m0 + at.row(0) + hit[j] < a.w.rows) {
      float z = 0.0f;
#pragma unroll
      for (int i = 0; i < S::I; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) z = hit[j] == (uint32_t)(i * 16 + r) ? acc[i][j][r] : z;
      a.hit[n0 + at.col(j)] = z;
    }
  }
  __syncthreads();
  if (threadIdx.x < S::N && n0 + threadIdx.x < a.x.rows) {
    float2 p = half[threadIdx.x];
#pragma unroll
    for (uint32_t k = 1; k < S::WM; ++k) {
      const float2 q = half[k * S::N + threadIdx.x];
      const float M = __builtin_fmaxf(p.x, q.x);
      p = float2{M, p.y * rescale(p.x, M) + q.y * rescale(q.x, M)};
    }
    a.part[(uint64_t)(n0 + threadIdx.x) * a.n_vt + vt] = p;
  }
  if constexpr (ROW) tile_row<S>(acc, a, m0, n0, a.rows + id);
}

// dz of the tile, in 16 bits (rounded to nearest: off by half a step of its
// own size, which the products average out), 0 for rows without a target and
// in the padding.  It passes through LDS, so that it is stored in whole rows of
// the tile.  Bound by the matrix cores: the two pieces of 4096 x 50304 x 2048 take
// 865 us of a trace on average (976 TFLOP/s; 943 us with the row), a tenth of it the
// exponentials and the store.
template <class T, class S, RowsAt AT, bool ROW>
__global__ void __launch_bounds__(S::kThreads) logit_dz_kernel(const LogitArgs a) {
  extern __shared__ __align__(16) unsigned char lds[];
  const uint32_t id = xcd_run(blockIdx.x, a.n_tiles, a.xcds);
  const uint32_t m0 = (id / a.nt) * S::M, n0 = (id % a.nt) * S::N;
  const Place<S> at;
  // what the epilogue needs of its tokens, in flight during the product
  float lse[S::J];
  uint32_t hit[S::J];
#pragma unroll
  for (int j = 0; j < S::J; ++j) {
    lse[j] = a.lse[min(n0 + at.col(j), a.x.rows - 1u)];
    hit[j] = target_from<S>(a, n0 + at.col(j), a.v0 + m0 + at.row(0));
  }
  f32x4 acc[S::I][S::J];
  gemm_tile<T, S, AT, false, false>(a.w, a.x, m0, n0, 0, a.K, lds, acc);
  if constexpr (ROW) tile_row<S>(acc, a, m0, n0, a.rows + id);
  uint16_t* st = reinterpret_cast<uint16_t*>(lds);
#pragma unroll
  for (int j = 0; j < S::J; ++j) {
    const bool live = hit[j] != kNoTarget;
#pragma unroll
    for (int i = 0; i < S::I; ++i) {
      uint32_t b[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float p = exp_of(acc[i][j][r] - lse[j]);
        p = (p - (hit[j] == (uint32_t)(i * 16 + r) ? 1.0f : 0.0f)) * T::kDzScale;
        b[r] = T::bits(live && m0 + at.row(i) + r < a.w.rows ? p : 0.0f);
      }
      *reinterpret_cast<uint2*>(st + at.col(j) * stage_row<S>() + at.row(i)) =
          uint2{b[0] | b[1] << 16, b[2] | b[3] << 16};
    }
  }
  __syncthreads();
  const uint32_t t = threadIdx.x, ch = t % (S::M / 8) * 8u;
#pragma unroll 4
  for (uint32_t k = t / (S::M / 8); k < S::N; k += S::kThreads / (S::M / 8)) {
    const uint32_t n = n0 + k, v = m0 + ch;
    if (n < a.x.rows && v < a.v_pad)
      *reinterpret_cast<u32x4*>(a.dz + (uint64_t)n * a.v_pad + v) =
          *reinterpret_cast<const u32x4*>(st + k * stage_row<S>() + ch);
  }
}

// ---- dx and dW --------------------------------------------------------------------

template <class T, class S, RowsAt AT>
__device__ __forceinline__ void dx_tile(const ProductArgs& a, uint32_t id, unsigned char* lds) {
  const uint32_t n0 = (id % a.nt) * S::N, rest = id / a.nt;
  const uint32_t m0 = (rest % a.md) * S::M, split = rest / a.md;
  const uint32_t k0 = split * a.chunk, k1 = min(k0 + a.chunk, a.rows);
  if (k0 >= k1 && !a.first) return;
  f32x4 acc[S::I][S::J];
  if (k0 < k1) {
    gemm_tile<T, S, AT, true, false>(a.w, a.dz, m0, n0, k0, k1, lds, acc);
  } else {
#pragma unroll
    for (int i = 0; i < S::I; ++i)
#pragma unroll
      for (int j = 0; j < S::J; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }
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
        if (m < a.d) {
          f32x4* q = reinterpret_cast<f32x4*>(p);
          *q = a.first ? acc[i][j] : *q + acc[i][j];
        }
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (m + r < a.d) p[r] = a.first ? acc[i][j][r] : p[r] + acc[i][j][r];
      }
    }
  }
}

template <class T, class S>
__device__ __forceinline__ void dw_tile(const ProductArgs& a, uint32_t id, unsigned char* lds) {
  const uint32_t m0 = (id % a.md) * S::M, n0 = (id / a.md) * S::N;
  const float g = *a.grad * (1.0f / T::kDzScale);
  f32x4 acc[S::I][S::J];
  gemm_tile<T, S, kAt16, true, true>(a.x, a.dz, m0, n0, 0, a.N, lds, acc);
  const Place<S> at;
  uint16_t* st = reinterpret_cast<uint16_t*>(lds);
#pragma unroll
  for (int j = 0; j < S::J; ++j)
#pragma unroll
    for (int i = 0; i < S::I; ++i) {
      uint32_t b[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) b[r] = T::bits(acc[i][j][r] * g);
      *reinterpret_cast<uint2*>(st + at.col(j) * stage_row<S>() + at.row(i)) =
          uint2{b[0] | b[1] << 16, b[2] | b[3] << 16};
    }
  __syncthreads();
  const uint32_t t = threadIdx.x, ch = t % (S::M / 8) * 8u;
#pragma unroll 4
  for (uint32_t k = t / (S::M / 8); k < S::N; k += S::kThreads / (S::M / 8)) {
    const uint32_t v = n0 + k, c = m0 + ch;
    if (v >= a.rows || c >= a.d) continue;
    uint16_t* p = a.dw + (uint64_t)v * a.d + c;
    const uint16_t* s = st + k * stage_row<S>() + ch;
    if (c + 8u <= a.d) {
      *reinterpret_cast<u32x4_at2*>(p) = *reinterpret_cast<const u32x4*>(s);
    } else {
      for (uint32_t e = 0; c + e < a.d; ++e) p[e] = s[e];
    }
  }
}

// Both products of dz (see ProductArgs).  dx's tile is dx^T (d down, tokens
// across) over a split of the piece, so a lane stores four fp32 of one token; dW's
// is dW^T over all tokens, stored through LDS in whole rows.  Bound by the matrix
// cores: 4096 x 50304 x 2048 takes 1537 us of a trace on average (1098 TFLOP/s); 16
// tokens x 128256 x 8192 963 us (4.4 TB/s: W read and dW written once).
template <class T, class S, RowsAt AT>
__global__ void __launch_bounds__(S::kThreads) products_kernel(const ProductArgs a) {
  extern __shared__ __align__(16) unsigned char lds[];
  if (blockIdx.x < a.n_dx) dx_tile<T, S, AT>(a, xcd_run(blockIdx.x, a.n_dx, a.xcds), lds);
  else dw_tile<T, S>(a, xcd_run(blockIdx.x - a.n_dx, a.n_dw, a.xcds), lds);
}

// f(type)
template <class F>
int32_t for_dtype(uint32_t dtype, F&& f) {
  return dtype == SDC_BF16 ? f(Bf16()) : f(Fp16());
}

// f(type, shape) of the logits' product; tile: rows of the shape.  kDeep has the
// shapes for few tokens, the others the square ones.
template <RowsAt AT, class F>
int32_t for_logits(uint32_t dtype, uint32_t tile, F&& f) {
  return for_dtype(dtype, [&](auto t) {
    if constexpr (AT == kDeep) return tile == 128 ? f(t, FewTile()) : f(t, FewTinyTile());
    else return tile == 256 ? f(t, BigTile()) : tile == 128 ? f(t, SmallTile()) : f(t, TinyTile());
  });
}

template <RowsAt AT>
int32_t launch_logit_lse(const HeadLaunch& h, const LogitArgs& a, hipStream_t s) {
  return for_logits<AT>(h.dtype, h.tile, [&](auto t, auto shape) {
    typedef decltype(t) T;
    typedef decltype(shape) S;
    const dim3 grid(a.n_tiles), block(S::kThreads);
    if (a.rows) hipLaunchKernelGGL((logit_lse_kernel<T, S, AT, true>), grid, block, S::kLds, s, a);
    else hipLaunchKernelGGL((logit_lse_kernel<T, S, AT, false>), grid, block, S::kLds, s, a);
    return launch_status();
  });
}

template <RowsAt AT>
int32_t launch_logit_dz(const HeadLaunch& h, const LogitArgs& a, hipStream_t s) {
  return for_logits<AT>(h.dtype, h.tile, [&](auto t, auto shape) {
    typedef decltype(t) T;
    typedef decltype(shape) S;
    const dim3 grid(a.n_tiles), block(S::kThreads);
    if (a.rows) hipLaunchKernelGGL((logit_dz_kernel<T, S, AT, true>), grid, block, lds_bytes<S>(), s, a);
    else hipLaunchKernelGGL((logit_dz_kernel<T, S, AT, false>), grid, block, lds_bytes<S>(), s, a);
    return launch_status();
  });
}

template <RowsAt AT>
int32_t launch_products(const HeadLaunch& h, const ProductArgs& x, hipStream_t s) {
  return for_dtype(h.dtype, [&](auto t) {
    const auto launch = [&](auto shape) {
      typedef decltype(t) T;
      typedef decltype(shape) S;
      hipLaunchKernelGGL((products_kernel<T, S, AT>), dim3(x.n_dx + x.n_dw), dim3(S::kThreads), lds_bytes<S>(), s, x);
      return launch_status();
    };
    return h.ptile == 256 ? launch(BigTile()) : launch(SmallTile());
  });
}

}  // namespace
}  // namespace sdc
