// attn_dq.hip -- the queries' gradient of softmax attention (csrc/attn.hip) for gfx950.
#include "attn_device.h"

namespace sdc {
namespace {

// One query's gradient by a wave: for the tiles that a mask cuts and that hold an infinity or
// NaN among their keys, where zero times what a masked key holds would not be zero.
template <class T>
__device__ __forceinline__ void dq_row(const AttnArgs& a, const Place32& p, uint32_t r) {
  const uint32_t lane = threadIdx.x & 63u;
  const int32_t t = (int32_t)token_of(a, r), lo = keys_begin(a, p, t), hi = keys_end(a, p, t);
  const uint64_t flat = flat_row(a, p, r);
  const unsigned char *q = query_row(a, p, r), *dout = a.dout + flat * (2u * a.d);
  const unsigned char *k = key_rows(a, p), *v = value_rows(a, p);
  const float l2 = a.l2[grouped_row(a, p, r)] + kPShift<T>, delta = a.delta[grouped_row(a, p, r)];
  float x[2] = {0.0f, 0.0f};
  for (int32_t k0 = lo; k0 < hi; k0 += 64) {
    const int32_t key = k0 + (int32_t)lane;
    float w = 0.0f;
    if (key < hi) {
      const float s = dot_rows<T>(q, k + (uint64_t)key * a.k_row, a.d);
      w = __builtin_amdgcn_exp2f(__builtin_fmaf(s, a.c, -l2)) *
          (dot_rows<T>(dout, v + (uint64_t)key * a.v_row, a.d) - delta);
    }
    const int32_t n = min(hi - k0, 64);
    for (int32_t j = 0; j < n; ++j) add_row<T>(x, __shfl(w, j), k + (uint64_t)(k0 + j) * a.k_row, a.d);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (lane + 64u * i < a.d) a.dq[flat * a.d + lane + 64u * i] = (uint16_t)T::bits(x[i] * a.scale);
}

// As the forward pass, a workgroup of W waves takes 32 W queries of a head of keys and
// streams the keys they attend past them.  A wave keeps its queries and their rows of
// dout in registers, and per block of 32 keys computes S^T = K Q^T and dP^T = V dout^T, the
// probabilities p = exp2(s c - lse log2(e)), dS = p (dP - delta), and adds K^T dS^T to
// dq^T.  dS is the one thing rounded to 16 bits on the way (off by half a step of its own
// size, which the sum over keys averages out).  Bound by the matrix cores, 62 % busy without a
// mask: 8192 tokens, 64/8 heads of 128 take 1460 us causal with delta's launch (1130 TFLOP/s of its three
// products).
template <class T, int DB, int W, bool ROW>
__global__ void __launch_bounds__(64 * W, W == 4 ? 2 : 1) attn_dq_kernel(const AttnArgs a) {
  extern __shared__ __align__(16) unsigned char lds[];
  __shared__ uint32_t found;  // an infinity or NaN among the keys of a tile that a mask cuts
  constexpr uint32_t kBytes = tile_bytes<DB>();
  const Place32 p = place_of<false>(a, blockIdx.x, 32u * W);
  Lane ln;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63u, half = lane >> 5;
  const uint32_t R = (uint32_t)p.lq * a.G, wg0 = p.tile * (32u * W), r0 = wg0 + wave * 32u;
  if (p.live && R != 0) {
    typename T::frag q[2 * DB], dout[2 * DB];
    const uint32_t r = r0 + (lane & 31u), c = min(r, R - 1u);
    const uint64_t flat = flat_row(a, p, c);
    load_row<T, DB>(query_row(a, p, c), r < R, a.d, q);
    load_row<T, DB>(a.dout + flat * (2u * a.d), r < R, a.d, dout);
    const float l2 = a.l2[grouped_row(a, p, c)], delta = a.delta[grouped_row(a, p, c)];
    // the lane's query attends keys [lo, lo + span)
    const int32_t mine = (int32_t)token_of(a, c), lo = keys_begin(a, p, mine);
    const uint32_t span = (uint32_t)max(keys_end(a, p, mine) - lo, 0);
    const auto token = [&](uint32_t x) SDC_INLINE { return (int32_t)token_of(a, min(x, R - 1u)); };
    const int32_t wg_begin = keys_begin(a, p, token(wg0)), wg_end = keys_end(a, p, token(wg0 + 32u * W - 1u));
    const int32_t begin = keys_begin(a, p, token(r0)), end = keys_end(a, p, token(r0 + 31u));
    const int32_t from = keys_begin(a, p, token(r0 + 31u)), to = keys_end(a, p, token(r0));
    const int32_t t0 = wg_begin / (int32_t)kAttnTile, t1 = (wg_end + (int32_t)kAttnTile - 1) / (int32_t)kAttnTile;
    const uint64_t first_score = flat * a.kw + 4u * half + 1u;  // of the lane's query, from 1
    const int shift = grad_shift<T>(a);
    const float f = power_of_two(shift - (int)kPShift<T>);
    f32x16 acc[DB];
#pragma unroll
    for (int m = 0; m < DB; ++m)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[m][e] = 0.0f;
    TileLoader<DB, W> lk, lv;
    lk.init(key_rows(a, p), a.k_row, a.d);
    lv.init(value_rows(a, p), a.v_row, a.d);
    const uint32_t lds0 = (uint32_t)(uintptr_t)(SDC_LDS unsigned char*)lds;
    TileReads<T> at(lds0);
    const auto fill = [&](int32_t t, uint32_t buf) SDC_INLINE {
      lk.fill((uint32_t)t * kAttnTile, (uint32_t)p.lk, lds0 + buf * (2u * kBytes));
      lv.fill((uint32_t)t * kAttnTile, (uint32_t)p.lk, lds0 + buf * (2u * kBytes) + kBytes);
    };
    if (t0 < t1) fill(t0, 0);
    // cut by a mask for some query of the workgroup
    const int32_t wg_from = keys_begin(a, p, token(wg0 + 32u * W - 1u)), wg_to = keys_end(a, p, token(wg0));
    if (threadIdx.x == 0) found = 0;
    uint32_t buf = 0;
    for (int32_t t = t0; t < t1; ++t, at.move(buf ? 0u - 2u * kBytes : 2u * kBytes), buf ^= 1u) {
      tile_barrier();  // this buffer is whole, and everyone has left the other
      if (t + 1 < t1) fill(t + 1, buf ^ 1u);
      const int32_t k0 = t * (int32_t)kAttnTile;
      if (k0 < wg_from || k0 + (int32_t)kAttnTile > wg_to) find_nonfinite<T, DB, W>(lds + buf * (2u * kBytes), &found);
      if (k0 >= end || k0 + (int32_t)kAttnTile <= begin) continue;
      const bool masked = k0 < from || k0 + (int32_t)kAttnTile > to;
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        f32x16 s, dp;
#pragma unroll
        for (int e = 0; e < 16; ++e) s[e] = dp[e] = 0.0f;
#pragma unroll
        for (int i = 0; i < 2 * DB; ++i) {
          s = mfma32(at.row(0, n, i), q[i], s);
          dp = mfma32(at.row(kBytes, n, i), dout[i], dp);
        }
        uint32_t first = (uint32_t)(k0 + 32 * n + 4 * (int32_t)half - lo);
        if constexpr (ROW) {
          if (masked) {
#pragma unroll
            for (int e = 0; e < 16; ++e) s[e] = first + element_row(e, 0) < span ? s[e] : 0.0f;
          }
          if (r < R) {
            ScoreSums c;
            add_scores(c, s, 0);
            join_scores(ln, c, first_score + (uint32_t)(k0 + 32 * n), 1u);
            if (c.odd != c.odd) ln.nf += nonfinite_scores(s);
          }
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float pr = __builtin_amdgcn_exp2f(__builtin_fmaf(s[e], a.c, -l2));
          s[e] = pr * (dp[e] - delta);
          if constexpr (kPShift<T> != 0.0f) s[e] *= f;
        }
        if (masked) {
          asm volatile("" : "+v"(first));  // so that this stays a branch: no selects for the other tiles
#pragma unroll
          for (int e = 0; e < 16; ++e)
            s[e] = first + element_row(e, 0) < span ? s[e] : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const typename T::frag w = operand<T>(s, i);
#pragma unroll
          for (int m = 0; m < DB; ++m) acc[m] = mfma32(at.column(0, m, 2 * n + i), w, acc[m]);
        }
      }
    }
    __syncthreads();  // found is
    if (found) {
      const uint32_t rows = min(r0 + 32u, R);
      for (uint32_t x = r0; x < rows; ++x) dq_row<T>(a, p, x);
    } else if (r < R) {
      const float g = a.scale * power_of_two(-shift);
      uint16_t* out = a.dq + flat * a.d;
#pragma unroll
      for (int m = 0; m < DB; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t x = 32u * m + 8u * e + 4u * half;
          if (x < a.d)
            store4<T>(out + x, acc[m][4 * e] * g, acc[m][4 * e + 1] * g, acc[m][4 * e + 2] * g, acc[m][4 * e + 3] * g);
        }
    }
  }
  if constexpr (ROW) store_tile_row<W>(ln, a.rows + blockIdx.x);
}

}  // namespace

int32_t launch_attn_dq(const AttnLaunch& l, const AttnArgs& a, hipStream_t s) {
  return for_dtype(l.dtype, [&](auto type) {
    typedef decltype(type) T;
    const auto launch = [&](auto db, auto waves) {
      constexpr int DB = decltype(db)::value, W = decltype(waves)::value;
      const dim3 grid(a.units), block(64 * W);
      constexpr uint32_t bytes = 4u * tile_bytes<DB>();
      if (a.rows) hipLaunchKernelGGL((attn_dq_kernel<T, DB, W, true>), grid, block, bytes, s, a);
      else hipLaunchKernelGGL((attn_dq_kernel<T, DB, W, false>), grid, block, bytes, s, a);
      return launch_status();
    };
    const auto shape = [&](auto db) {
      return l.waves == 1 ? launch(db, std::integral_constant<int, 1>()) : launch(db, std::integral_constant<int, 4>());
    };
    return a.d <= 64   ? shape(std::integral_constant<int, 2>())
           : a.d <= 96 ? shape(std::integral_constant<int, 3>())
                       : shape(std::integral_constant<int, 4>());
  });
}

}  // namespace sdc
