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

// A workgroup of W waves takes 32 W queries of a head of keys, a wave 32 of them, and
// streams the keys they attend past them in tiles of 64 (two buffers in LDS, the next
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
// Two loops in one another, the outer for the tiles that raise a reference: the inner one,
// which nearly all tiles take, then has no branch around the sums of values, which would cost
// a copy of them each time (8192 tokens, causal: 1163 us against 1218 when it was built).
//
// Bound by the matrix cores and the vector units beside them, which two waves a SIMD overlap
// (8192 tokens, 64/8 heads of 128: 1041 us causal, 2017 us and 1090 TFLOP/s without a mask,
// the matrix cores 53 % busy).  Waves of 64 queries, which read LDS half as
// often but leave one wave a SIMD, measured 20 to 50 % slower; the next tile's scores between
// this one's exponentials and products, which takes two sets of scores in registers, 45 %.
//
// Few queries, one wave: one buffer, so that four workgroups or more fit a CU and cover each
// other's loads (8 x 1 query of 32/8 heads against 8191 keys, this launch: 59 us with two buffers, 55 with one).
//
// SPLIT: the keys in a.splits parts, each leaving its unscaled sums, m and l.
constexpr float kFarOut = 0x1p27f;

template <class T, int DB, int W, bool ROW, bool SPLIT>
__global__ void __launch_bounds__(64 * W, 2) attn_kernel(const AttnArgs a) {
  extern __shared__ __align__(16) unsigned char lds[];
  __shared__ uint32_t found;  // an infinity or NaN among the values of a tile that a mask cuts
  constexpr uint32_t kBytes = tile_bytes<DB>();
  constexpr int32_t kTile = (int32_t)kAttnTile;
  constexpr bool kTwo = W > 1;  // buffers
  const uint32_t unit = SPLIT ? blockIdx.x / a.splits : blockIdx.x, split = SPLIT ? blockIdx.x % a.splits : 0u;
  const Place32 p = place_of<false>(a, unit, 32u * W);
  Lane ln;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63u, half = lane >> 5;
  const uint32_t R = (uint32_t)p.lq * a.G, wg0 = p.tile * (32u * W), r0 = wg0 + wave * 32u;
  if (p.live && R != 0) {
    const uint32_t r = r0 + (lane & 31u), mine = min(r, R - 1u);
    typename T::frag q[2 * DB];
    load_row<T, DB>(query_row(a, p, mine), r < R, a.d, q);
    const auto token = [&](uint32_t x) SDC_INLINE { return (int32_t)token_of(a, min(x, R - 1u)); };
    // the lane's query attends keys [lo, lo + span)
    const int32_t lo = keys_begin(a, p, token(mine));
    const uint32_t span = (uint32_t)max(keys_end(a, p, token(mine)) - lo, 0);
    // keys of the workgroup's, and of the wave's, queries: [begin, end), all attend [from, to)
    const int32_t wg_begin = keys_begin(a, p, token(wg0)), wg_end = keys_end(a, p, token(wg0 + 32u * W - 1u));
    const int32_t begin = keys_begin(a, p, token(r0)), end = keys_end(a, p, token(r0 + 31u));
    const int32_t from = keys_begin(a, p, token(r0 + 31u)), to = keys_end(a, p, token(r0));
    int32_t t0 = wg_begin / kTile, t1 = max((wg_end + kTile - 1) / kTile, t0);
    if constexpr (SPLIT) {
      const int32_t each = (t1 - t0 + (int32_t)a.splits - 1) / (int32_t)a.splits;
      t0 = min(t0 + (int32_t)split * each, t1);
      t1 = min(t0 + each, t1);
    }
    f32x16 o[DB];
#pragma unroll
    for (int m = 0; m < DB; ++m)
#pragma unroll
      for (int e = 0; e < 16; ++e) o[m][e] = 0.0f;
    float top = -__builtin_inff(), base = 0.0f, off = 0.0f, l = 0.0f;  // m, base, d (0 far out), sum of exponentials
    const float rise = 8.0f / a.c;
    const uint64_t first_score = flat_row(a, p, mine) * a.kw + 4u * half + 1u;  // of the lane's query, from 1
    TileLoader<DB, W> lk, lv;
    lk.init(key_rows(a, p), a.k_row, a.d);
    lv.init(value_rows(a, p), a.v_row, a.d);
    const uint32_t lds0 = (uint32_t)(uintptr_t)(SDC_LDS unsigned char*)lds;
    TileReads<T> at(lds0);
    uint32_t buf = 0;
    const auto fill = [&](int32_t t, uint32_t to_buf) SDC_INLINE {
      lk.fill((uint32_t)(t * kTile), (uint32_t)p.lk, lds0 + to_buf * (2u * kBytes));
      lv.fill((uint32_t)(t * kTile), (uint32_t)p.lk, lds0 + to_buf * (2u * kBytes) + kBytes);
    };
    // cut by a mask for some query of the workgroup
    const int32_t wg_from = keys_begin(a, p, token(wg0 + 32u * W - 1u)), wg_to = keys_end(a, p, token(wg0));
    if (threadIdx.x == 0) found = 0;
    // On to tile t: this buffer is whole, everyone has left the other, the next is filled.
    // One buffer: the wave has left it; its own loads fill it.
    const auto enter = [&](int32_t t) SDC_INLINE {
      if constexpr (kTwo) {
        tile_barrier();
        if (t + 1 < t1) fill(t + 1, buf ^ 1u);
      } else {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        fill(t, 0);
        tile_barrier();
      }
      if (t * kTile < wg_from || t * kTile + kTile > wg_to)
        find_nonfinite<T, DB, W>(lds + buf * (2u * kBytes) + kBytes, &found);
    };
    const auto leave = [&]() SDC_INLINE {
      if constexpr (kTwo) {
        at.move(buf ? 0u - 2u * kBytes : 2u * kBytes);
        buf ^= 1u;
      }
    };
    // A tile's scores, what the row takes of them, the masked ones as -inf; the largest of
    // the lane's query.
    f32x16 s[2];
    const auto scores = [&](int32_t t) SDC_INLINE {
      const int32_t k0 = t * kTile;
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 16; ++e) s[n][e] = 0.0f;
#pragma unroll
      for (int i = 0; i < 2 * DB; ++i)
#pragma unroll
        for (int n = 0; n < 2; ++n) s[n] = mfma32(at.row(0, n, i), q[i], s[n]);
      const bool cut = k0 < from || k0 + kTile > to;  // by a mask, for some query of the wave
      const uint32_t first = (uint32_t)(k0 + 4 * (int32_t)half - lo);
      const auto mask = [&](float with) SDC_INLINE {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 16; ++e) s[n][e] = first + 32u * n + element_row(e, 0) < span ? s[n][e] : with;
      };
      if constexpr (ROW) {
        if (cut) mask(0.0f);
        if (r < R) {
          ScoreSums c;
          add_scores(c, s[0], 0);
          add_scores(c, s[1], 1);
          join_scores(ln, c, first_score + (uint32_t)k0, 1u);
          if (c.odd != c.odd) ln.nf += nonfinite_scores(s[0]) + nonfinite_scores(s[1]);
        }
      }
      if (cut) mask(-__builtin_inff());
      float most = s[0][0];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 16; ++e) most = __builtin_fmaxf(most, s[n][e]);
      return both_max(most);
    };
    // the wave's own tiles, [tw, te), and before and after them those of others of the workgroup
    t0 = uniform(t0);
    t1 = uniform(t1);
    const int32_t te = uniform(min(max((end + kTile - 1) / kTile, t0), t1));
    const int32_t tw = uniform(min(max(begin / kTile, t0), te));
    if (kTwo && t0 < t1) fill(t0, 0);
    int32_t t = t0;
    for (; t < tw; ++t) {
      enter(t);
      leave();
    }
    float most = 0.0f;
    if (t < te) {
      enter(t);
      most = scores(t);
    }
    while (t < te) {
      const float was = top, before = off;
      top = most > was + rise ? most : was;
      base = top == -__builtin_inff() ? 0.0f : top * a.c;
      const bool near = __builtin_fabsf(base) < kFarOut, far_out = __any(!near);
      off = top != -__builtin_inff() && near ? __builtin_fmaf(top, a.c, -base) : 0.0f;
      const float f = was == top ? 1.0f : __builtin_amdgcn_exp2f((was - top) * a.c - before + off);
      l *= f;
#pragma unroll
      for (int m = 0; m < DB; ++m)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[m][e] *= f;
      do {
        if (!far_out) {
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 16; ++e) s[n][e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n][e], a.c, -base));
        } else {
          const float m = top == -__builtin_inff() ? 0.0f : top;
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 16; ++e) s[n][e] = __builtin_amdgcn_exp2f((s[n][e] - m) * a.c + off);
        }
        float sum = 0.0f;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 16; ++e) sum += s[n][e];
        l += sum;
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const typename T::frag w = operand<T>(s[i >> 1], i & 1);
#pragma unroll
          for (int m = 0; m < DB; ++m) o[m] = mfma32(at.column(kBytes, m, i), w, o[m]);
        }
        __builtin_amdgcn_s_setprio(0);
        leave();
        if (++t >= te) break;
        enter(t);
        most = scores(t);
      } while (!__any(most > top + rise));
    }
    for (; t < t1; ++t) {
      enter(t);
      leave();
    }
    const float sum = both_sum(l);
    __syncthreads();  // found is
    if (found) {
      const uint32_t rows = min(r0 + 32u, R);
      for (uint32_t x = r0; x < rows; ++x) attn_row<T, SPLIT>(a, p, x, t0 * kTile, t1 * kTile, split);
    } else if (r < R) {
      // a query that attends nothing: out 0, lse -inf
      const bool none = top == -__builtin_inff() && !(sum != sum);
      const uint64_t row = SPLIT ? grouped_row(a, p, r) * a.splits + split : flat_row(a, p, r);
      const float f = SPLIT ? __builtin_amdgcn_exp2f(-off) : none ? 0.0f : 1.0f / sum;  // SPLIT: from base to m c
      if (half == 0) {
        if constexpr (SPLIT) a.part_ml[row] = float2{top, sum * f};
        else a.lse[row] = none ? -__builtin_inff() : log_sum(top, a.scale, sum, off);
      }
#pragma unroll
      for (int m = 0; m < DB; ++m)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const uint32_t e = 32u * m + 8u * g + 4u * half;
          if (e >= a.d) continue;
          const f32x4 x = {o[m][4 * g] * f, o[m][4 * g + 1] * f, o[m][4 * g + 2] * f, o[m][4 * g + 3] * f};
          if constexpr (SPLIT) *reinterpret_cast<f32x4*>(a.part + row * a.d + e) = x;
          else store4<T>(a.out + row * a.d + e, x.x, x.y, x.z, x.w);
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
  // the splits' factors, one a lane (at most 64)
  const float2 ml = lane < a.splits ? a.part_ml[at + lane] : float2{-__builtin_inff(), 0.0f};
  float top = ml.x;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, o));
  const float m = top == -__builtin_inff() ? 0.0f : top;
  const float mine = __builtin_amdgcn_exp2f((ml.x - m) * a.c);
  float x[2] = {0.0f, 0.0f}, sum = 0.0f;
  for (uint32_t k = 0; k < a.splits; k += 8) {  // eight splits' loads in flight
    float v[8][2];
#pragma unroll
    for (uint32_t j = 0; j < 8; ++j)
#pragma unroll
      for (uint32_t i = 0; i < 2; ++i)
        v[j][i] = k + j < a.splits && lane + 64u * i < a.d ? a.part[(at + k + j) * a.d + lane + 64u * i] : 0.0f;
#pragma unroll
    for (uint32_t j = 0; j < 8; ++j) {
      if (k + j >= a.splits) break;
      const float f = __shfl(mine, k + j);
      sum += __shfl(ml.y, k + j) * f;
#pragma unroll
      for (uint32_t i = 0; i < 2; ++i) x[i] += v[j][i] * f;
    }
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
    const auto launch = [&](auto db, auto waves) {
      constexpr int DB = decltype(db)::value, W = decltype(waves)::value;
      const dim3 grid(a.units * a.splits), block(64 * W);
      constexpr uint32_t bytes = (W > 1 ? 4u : 2u) * tile_bytes<DB>();
      const bool split = a.splits > 1;
      if (a.rows && split) hipLaunchKernelGGL((attn_kernel<T, DB, W, true, true>), grid, block, bytes, s, a);
      else if (a.rows) hipLaunchKernelGGL((attn_kernel<T, DB, W, true, false>), grid, block, bytes, s, a);
      else if (split) hipLaunchKernelGGL((attn_kernel<T, DB, W, false, true>), grid, block, bytes, s, a);
      else hipLaunchKernelGGL((attn_kernel<T, DB, W, false, false>), grid, block, bytes, s, a);
      return launch_status();
    };
    const auto shape = [&](auto db) {
      return l.waves == 1 ? launch(db, std::integral_constant<int, 1>()) : launch(db, std::integral_constant<int, 4>());
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
