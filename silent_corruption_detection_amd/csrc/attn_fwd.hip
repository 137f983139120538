// attn_fwd.hip -- the forward pass of softmax attention (csrc/attn.hip) for gfx950.
#include "attn_device.h"

namespace sdc {
namespace {

// lse from the largest score (or one near it) and the sum of exponentials less its reference.
__device__ __forceinline__ float log_sum(float top, float scale, float sum, float off) {
  return __builtin_fmaf(top, scale, (__builtin_amdgcn_logf(sum) - off) * kLn2);
}

// One query by a wave, over the keys it attends in [first, last): for the tiles that a mask
// cuts and that hold an infinity or NaN among their values, where zero times what a masked
// key holds would not be zero.
template <class T, bool SPLIT>
__device__ __forceinline__ void attn_row(const AttnArgs& a, const Place32& p, uint32_t r, int32_t first, int32_t last,
                                         uint32_t split) {
  const uint32_t lane = threadIdx.x & 63u;
  const int32_t t = (int32_t)token_of(a, r), lo = max(keys_begin(a, p, t), first), hi = min(keys_end(a, p, t), last);
  const unsigned char *q = query_row(a, p, r), *k = key_rows(a, p), *v = value_rows(a, p);
  float top = -__builtin_inff();
  for (int32_t k0 = lo; k0 < hi; k0 += 64) {
    const int32_t key = k0 + (int32_t)lane;
    if (key < hi) top = __builtin_fmaxf(top, dot_rows<T>(q, k + (uint64_t)key * a.k_row, a.d));
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, o));
  const float m = top == -__builtin_inff() ? 0.0f : top;
  float sum = 0.0f, x[2] = {0.0f, 0.0f};
  for (int32_t k0 = lo; k0 < hi; k0 += 64) {
    const int32_t key = k0 + (int32_t)lane;
    float w = 0.0f;
    if (key < hi) w = __builtin_amdgcn_exp2f((dot_rows<T>(q, k + (uint64_t)key * a.k_row, a.d) - m) * a.c);
    sum += w;
    const int32_t n = min(hi - k0, 64);
    for (int32_t j = 0; j < n; ++j) add_row<T>(x, __shfl(w, j), v + (uint64_t)(k0 + j) * a.v_row, a.d);
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
  const bool none = top == -__builtin_inff() && !(sum != sum);
  const uint64_t row = SPLIT ? grouped_row(a, p, r) * a.splits + split : flat_row(a, p, r);
  if (lane == 0) {
    if constexpr (SPLIT) a.part_ml[row] = float2{top, sum};
    else a.lse[row] = none ? -__builtin_inff() : log_sum(top, a.scale, sum, 0.0f);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (lane + 64u * i >= a.d) continue;
    if constexpr (SPLIT) a.part[row * a.d + lane + 64u * i] = x[i];
    else a.out[row * a.d + lane + 64u * i] = (uint16_t)T::bits(none ? 0.0f : x[i] / sum);
  }
}

// A workgroup of W waves takes 32 QB W queries of a head of keys, a wave 32 QB of them,
// and streams the keys they attend past them in tiles of 64 (two buffers in LDS, the next
// filled by direct loads while this one is multiplied).  The queries stay in registers, as
// do the sums of values: out^T = V^T P^T with a query per lane, so its rescaling is one
// factor a lane.
//
// The softmax runs on exponents s c, c = scale log2(e), less a reference: base, the rounded
// product of c and a score m that a query raises only when a tile's maximum passes it by
// more than 8 / c.  Probabilities are then at most 2^8, sums in fp32 are none the worse, and
// most tiles rescale nothing.  s c - base is one fused operation, exact but for its own
// rounding, so that base's rounding is no error but a factor 2^d, d = m c - base, that out's
// sums and l share.  From |base| of 2^27 on (kFarOut) that factor could overflow: there the
// difference of scores comes first and the reference is m c itself.
//
// SPLIT: the keys in a.splits parts, each leaving its unscaled sums, m and l.
constexpr float kFarOut = 0x1p27f;

template <class T, int DB, int W, int QB, bool ROW, bool SPLIT>
__global__ void __launch_bounds__(64 * W, W * QB == 4 ? 2 : 1) attn_kernel(const AttnArgs a) {
  extern __shared__ __align__(16) unsigned char lds[];
  constexpr uint32_t kBytes = tile_bytes<DB>();
  const uint32_t unit = SPLIT ? blockIdx.x / a.splits : blockIdx.x, split = SPLIT ? blockIdx.x % a.splits : 0u;
  const Place32 p = place_of<false>(a, unit, 32u * QB * W);
  Lane ln;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63u, half = lane >> 5;
  const uint32_t R = (uint32_t)p.lq * a.G, wg0 = p.tile * (32u * QB * W), r0 = wg0 + wave * (32u * QB);
  if (p.live && R != 0) {
    typename T::frag q[QB][2 * DB];
    int32_t lo[QB], hi[QB];
#pragma unroll
    for (int b = 0; b < QB; ++b) {
      const uint32_t r = r0 + 32u * b + (lane & 31u), c = min(r, R - 1u);
      load_row<T, DB>(query_row(a, p, c), r < R, a.d, q[b]);
      const int32_t t = (int32_t)token_of(a, c);
      lo[b] = keys_begin(a, p, t);
      hi[b] = keys_end(a, p, t);
    }
    // keys of the workgroup's, and of the wave's, queries: [begin, end), all attend [from, to)
    const auto token = [&](uint32_t r) SDC_INLINE { return (int32_t)token_of(a, min(r, R - 1u)); };
    const int32_t wg_begin = keys_begin(a, p, token(wg0)), wg_end = keys_end(a, p, token(wg0 + 32u * QB * W - 1u));
    const int32_t begin = keys_begin(a, p, token(r0)), end = keys_end(a, p, token(r0 + 32u * QB - 1u));
    const int32_t from = keys_begin(a, p, token(r0 + 32u * QB - 1u)), to = keys_end(a, p, token(r0));
    int32_t t0 = wg_begin / (int32_t)kAttnTile, t1 = max((wg_end + (int32_t)kAttnTile - 1) / (int32_t)kAttnTile, t0);
    if constexpr (SPLIT) {
      const int32_t each = (t1 - t0 + (int32_t)a.splits - 1) / (int32_t)a.splits;
      t0 = min(t0 + (int32_t)split * each, t1);
      t1 = min(t0 + each, t1);
    }
    f32x16 o[QB][DB];
    float top[QB], base[QB], off[QB], l[QB];  // m, base, d (0 far out) and the sum of exponentials
#pragma unroll
    for (int b = 0; b < QB; ++b) {
      top[b] = -__builtin_inff();
      base[b] = off[b] = l[b] = 0.0f;
#pragma unroll
      for (int m = 0; m < DB; ++m)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[b][m][e] = 0.0f;
    }
    const float rise = 8.0f / a.c;
    uint64_t first_score[QB];  // of the lane's query, from 1
#pragma unroll
    for (int b = 0; b < QB; ++b)
      first_score[b] = flat_row(a, p, min(r0 + 32u * b + (lane & 31u), R - 1u)) * a.kw + 4u * half + 1u;
    // the tile's part of the row; has: which of the scores attend (cut tiles)
    const auto score_row = [&](int b, const f32x16 (&z)[2], int32_t k0, bool all, const uint32_t (&has)[2])
                               SDC_INLINE {
      if (r0 + 32u * b + (lane & 31u) >= R) return;
      ScoreSums c;
#pragma unroll
      for (int n = 0; n < 2; ++n) add_scores(c, z[n], n, all, has[n]);
      join_scores(ln, c, first_score[b] + (uint32_t)k0, 1u);
      if (c.odd != c.odd) ln.nf += nonfinite_scores(z[0], all, has[0]) + nonfinite_scores(z[1], all, has[1]);
    };
    TileLoader<DB, W> lk, lv;
    lk.init(key_rows(a, p), a.k_row, a.d);
    lv.init(value_rows(a, p), a.v_row, a.d);
    const uint32_t lds0 = (uint32_t)(uintptr_t)(SDC_LDS unsigned char*)lds;
    TileReads<T> at(lds0);
    const auto fill = [&](int32_t t, uint32_t buf) SDC_INLINE {
      lk.fill((uint32_t)t * kAttnTile, (uint32_t)p.lk, lds0 + buf * (2u * kBytes));
      lv.fill((uint32_t)t * kAttnTile, (uint32_t)p.lk, lds0 + buf * (2u * kBytes) + kBytes);
    };
    t0 = uniform(t0);
    t1 = uniform(t1);
    if (t0 < t1) fill(t0, 0);
    bool redo = false;
    uint32_t buf = 0;
    // On to tile t: this buffer is whole, everyone has left the other, the next is filled.
    const auto enter = [&](int32_t t) SDC_INLINE {
      tile_barrier();
      if (t + 1 < t1) fill(t + 1, buf ^ 1u);
    };
    const auto leave = [&]() SDC_INLINE {
      at.move(buf ? 0u - 2u * kBytes : 2u * kBytes);
      buf ^= 1u;
    };
    // the wave's own tiles, [tw, te), and before and after them those of others of the workgroup
    const int32_t te = uniform(min(max((end + (int32_t)kAttnTile - 1) / (int32_t)kAttnTile, t0), t1));
    const int32_t tw = uniform(min(max(begin / (int32_t)kAttnTile, t0), te));
    int32_t t = t0;
    for (; t < tw; ++t) {
      enter(t);
      leave();
    }
    // Two loops in one another, the outer for the tiles that raise a reference: the inner
    // one, which nearly all tiles take, then has no branch around the sums of values, which
    // would cost a copy of them each time.  An inner turn goes from a tile's scores to the next's.
    f32x16 s[QB][2];
    float most[QB];
    const auto scores = [&]() SDC_INLINE {
      const int32_t k0 = t * (int32_t)kAttnTile;
#pragma unroll
      for (int b = 0; b < QB; ++b)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 16; ++e) s[b][n][e] = 0.0f;
#pragma unroll
      for (int i = 0; i < 2 * DB; ++i)
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const typename T::frag f = at.row(0, n, i);
#pragma unroll
          for (int b = 0; b < QB; ++b) s[b][n] = mfma32(f, q[b][i], s[b][n]);
        }
      if (k0 < from || k0 + (int32_t)kAttnTile > to) {  // cut by a mask for some query
#pragma unroll
        for (int b = 0; b < QB; ++b) {
          const uint32_t first = (uint32_t)(k0 + 4 * (int32_t)half - lo[b]), all = (uint32_t)max(hi[b] - lo[b], 0);
          uint32_t has[2] = {0, 0};
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 16; ++e) has[n] |= first + 32u * n + element_row(e, 0) < all ? 1u << e : 0u;
          if constexpr (ROW) score_row(b, s[b], k0, false, has);
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 16; ++e) s[b][n][e] = has[n] >> e & 1u ? s[b][n][e] : -__builtin_inff();
        }
        redo |= tile_nonfinite<T, DB>(lds + buf * (2u * kBytes) + kBytes);
      } else if constexpr (ROW) {
        const uint32_t has[2] = {0xFFFFu, 0xFFFFu};
#pragma unroll
        for (int b = 0; b < QB; ++b) score_row(b, s[b], k0, true, has);
      }
#pragma unroll
      for (int b = 0; b < QB; ++b) {
        most[b] = s[b][0][0];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 16; ++e) most[b] = __builtin_fmaxf(most[b], s[b][n][e]);
        most[b] = both_max(most[b]);
      }
    };
    if (t < te) {
      enter(t);
      scores();
    }
    while (t < te) {
      bool far_out = false;
#pragma unroll
      for (int b = 0; b < QB; ++b) {
        const float was = top[b], before = off[b];
        top[b] = most[b] > was + rise ? most[b] : was;
        base[b] = top[b] == -__builtin_inff() ? 0.0f : top[b] * a.c;
        const bool near = __builtin_fabsf(base[b]) < kFarOut;
        off[b] = top[b] != -__builtin_inff() && near ? __builtin_fmaf(top[b], a.c, -base[b]) : 0.0f;
        const float f = was == top[b] ? 1.0f : __builtin_amdgcn_exp2f((was - top[b]) * a.c - before + off[b]);
        far_out |= __any(!near);
        l[b] *= f;
#pragma unroll
        for (int m = 0; m < DB; ++m)
#pragma unroll
          for (int e = 0; e < 16; ++e) o[b][m][e] *= f;
      }
      bool raise;
      do {
#pragma unroll
        for (int b = 0; b < QB; ++b) {
          if (!far_out) {
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int e = 0; e < 16; ++e)
                s[b][n][e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[b][n][e], a.c, -base[b]));
          } else {
            const float m = top[b] == -__builtin_inff() ? 0.0f : top[b];
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int e = 0; e < 16; ++e) s[b][n][e] = __builtin_amdgcn_exp2f((s[b][n][e] - m) * a.c + off[b]);
          }
          float sum = 0.0f;
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 16; ++e) sum += s[b][n][e];
          l[b] += sum;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          typename T::frag w[QB];
#pragma unroll
          for (int b = 0; b < QB; ++b) w[b] = operand<T>(s[b][i >> 1], i & 1);
#pragma unroll
          for (int m = 0; m < DB; ++m) {
            const typename T::frag f = at.column(kBytes, m, i);
#pragma unroll
            for (int b = 0; b < QB; ++b) o[b][m] = mfma32(f, w[b], o[b][m]);
          }
        }
        leave();
        if (++t >= te) break;
        enter(t);
        scores();
        raise = false;
#pragma unroll
        for (int b = 0; b < QB; ++b) raise |= __any(most[b] > top[b] + rise);
      } while (!raise);
    }
    for (; t < t1; ++t) {
      enter(t);
      leave();
    }
    if (redo) {
      const uint32_t rows = min(r0 + 32u * QB, R);
      for (uint32_t r = r0; r < rows; ++r)
        attn_row<T, SPLIT>(a, p, r, t0 * (int32_t)kAttnTile, t1 * (int32_t)kAttnTile, split);
    } else {
#pragma unroll
      for (int b = 0; b < QB; ++b) {
        const uint32_t r = r0 + 32u * b + (lane & 31u);
        const float sum = both_sum(l[b]);
        if (r >= R) continue;
        if constexpr (SPLIT) {
          const uint64_t row = grouped_row(a, p, r) * a.splits + split;
          const float f = __builtin_amdgcn_exp2f(-off[b]);  // from base to m c
          if (half == 0) a.part_ml[row] = float2{top[b], sum * f};
          float* out = a.part + row * a.d;
#pragma unroll
          for (int m = 0; m < DB; ++m)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              const uint32_t e = 32u * m + 8u * g + 4u * half;
              if (e < a.d)
                *reinterpret_cast<f32x4*>(out + e) =
                    f32x4{o[b][m][4 * g] * f, o[b][m][4 * g + 1] * f, o[b][m][4 * g + 2] * f, o[b][m][4 * g + 3] * f};
            }
        } else {
          // a query that attends nothing: out 0, lse -inf
          const bool none = top[b] == -__builtin_inff() && !(sum != sum);
          const float f = none ? 0.0f : 1.0f / sum;
          const uint64_t row = flat_row(a, p, r);
          if (half == 0) a.lse[row] = none ? -__builtin_inff() : log_sum(top[b], a.scale, sum, off[b]);
          uint16_t* out = a.out + row * a.d;
#pragma unroll
          for (int m = 0; m < DB; ++m)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              const uint32_t e = 32u * m + 8u * g + 4u * half;
              if (e < a.d)
                store4<T>(out + e, o[b][m][4 * g] * f, o[b][m][4 * g + 1] * f, o[b][m][4 * g + 2] * f,
                          o[b][m][4 * g + 3] * f);
            }
        }
      }
    }
  }
  if constexpr (ROW) store_tile_row<W>(ln, a.rows + blockIdx.x);
}

// Joins the splits of a row: out = sum_k f_k o_k / sum_k f_k l_k with f_k = 2^((m_k - m) c), in
// split order.  A wave per row; rows outside every sequence have none.
template <class T>
__global__ void __launch_bounds__(256) attn_join_kernel(const AttnArgs a, uint64_t rows) {
  const uint32_t lane = threadIdx.x & 63u;
  const uint64_t n = (uint64_t)blockIdx.x * 4u + (threadIdx.x >> 6);  // of [rows][hq]
  if (n >= rows * a.hq) return;
  const uint64_t row = n / a.hq;
  const uint32_t head = (uint32_t)(n % a.hq);
  if (a.seq_q && !in_sequences(a.seq_q, a.batch, a.len_q, (uint32_t)row)) return;
  const uint64_t at = ((head / a.G) * rows * a.G + row * a.G + head % a.G) * a.splits;
  float top = -__builtin_inff(), sum = 0.0f;
  for (uint32_t k = 0; k < a.splits; ++k) top = __builtin_fmaxf(top, a.part_ml[at + k].x);
  const float m = top == -__builtin_inff() ? 0.0f : top;
  float x[2] = {0.0f, 0.0f};
#pragma unroll 4
  for (uint32_t k = 0; k < a.splits; ++k) {
    const float2 ml = a.part_ml[at + k];
    const float f = __builtin_amdgcn_exp2f((ml.x - m) * a.c);
    sum += ml.y * f;
    const float* part = a.part + (at + k) * a.d;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (lane + 64u * i < a.d) x[i] += part[lane + 64u * i] * f;
  }
  const bool none = top == -__builtin_inff() && !(sum != sum);
  if (lane == 0) a.lse[n] = none ? -__builtin_inff() : log_sum(top, a.scale, sum, 0.0f);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (lane + 64u * i < a.d) a.out[n * a.d + lane + 64u * i] = (uint16_t)T::bits(none ? 0.0f : x[i] / sum);
}

}  // namespace

int32_t launch_attn(const AttnLaunch& l, const AttnArgs& a, hipStream_t s) {
  return for_dtype(l.dtype, [&](auto type) {
    typedef decltype(type) T;
    const auto launch = [&](auto db, auto waves, auto blocks) {
      constexpr int DB = decltype(db)::value, W = decltype(waves)::value, QB = decltype(blocks)::value;
      const dim3 grid(a.units * a.splits), block(64 * W);
      constexpr uint32_t bytes = 4u * tile_bytes<DB>();
      const bool split = a.splits > 1;
      if (a.rows && split) hipLaunchKernelGGL((attn_kernel<T, DB, W, QB, true, true>), grid, block, bytes, s, a);
      else if (a.rows) hipLaunchKernelGGL((attn_kernel<T, DB, W, QB, true, false>), grid, block, bytes, s, a);
      else if (split) hipLaunchKernelGGL((attn_kernel<T, DB, W, QB, false, true>), grid, block, bytes, s, a);
      else hipLaunchKernelGGL((attn_kernel<T, DB, W, QB, false, false>), grid, block, bytes, s, a);
      return launch_status();
    };
    const auto shape = [&](auto db) {
      std::integral_constant<int, 1> one;
      if (l.waves == 1) return launch(db, one, one);
      if (l.blocks == 2) return launch(db, std::integral_constant<int, 4>(), std::integral_constant<int, 2>());
      return launch(db, std::integral_constant<int, 4>(), one);
    };
    int32_t st = a.d <= 64   ? shape(std::integral_constant<int, 2>())
                 : a.d <= 96 ? shape(std::integral_constant<int, 3>())
                             : shape(std::integral_constant<int, 4>());
    if (st || a.splits == 1) return st;
    const uint64_t rows = a.seq_q ? a.len_q : (uint64_t)a.batch * a.len_q;
    hipLaunchKernelGGL(attn_join_kernel<T>, dim3((uint32_t)((rows * a.hq + 3) / 4)), dim3(256), 0, s, a, rows);
    return launch_status();
  });
}

}  // namespace sdc
