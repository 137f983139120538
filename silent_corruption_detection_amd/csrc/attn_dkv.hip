// attn_dkv.hip -- the keys' and values' gradients of softmax attention (csrc/attn.hip)
// for gfx950.
#include "attn_device.h"

namespace sdc {
namespace {

// One key's and value's gradient by a wave, over the queries [first, last): for the tiles
// that a mask cuts and that hold an infinity or NaN among their queries or rows of dout, where
// zero times what a masked query holds would not be zero.  row: of dk and dv; part: the
// split's first row.
template <class T, bool SPLIT>
__device__ __forceinline__ void dkv_row(const AttnArgs& a, const Place32& p, int32_t key, int32_t first, int32_t last,
                                        uint64_t row, uint64_t part) {
  const uint32_t lane = threadIdx.x & 63u;
  const unsigned char *k = key_rows(a, p) + (uint64_t)key * a.k_row, *v = value_rows(a, p) + (uint64_t)key * a.v_row;
  const auto dout = [&](int32_t r) SDC_INLINE { return a.dout + flat_row(a, p, (uint32_t)r) * (2u * a.d); };
  float xk[2] = {0.0f, 0.0f}, xv[2] = {0.0f, 0.0f};
  for (int32_t q0 = first; q0 < last; q0 += 64) {
    const int32_t r = q0 + (int32_t)lane;
    float w = 0.0f, dw = 0.0f;
    if (r < last) {
      const float s = dot_rows<T>(query_row(a, p, (uint32_t)r), k, a.d);
      w = __builtin_amdgcn_exp2f(__builtin_fmaf(s, a.c, -(a.l2[grouped_row(a, p, (uint32_t)r)] + kPShift<T>)));
      dw = w * (dot_rows<T>(dout(r), v, a.d) - a.delta[grouped_row(a, p, (uint32_t)r)]);
    }
    const int32_t n = min(last - q0, 64);
    for (int32_t j = 0; j < n; ++j) {
      add_row<T>(xv, __shfl(w, j), dout(q0 + j), a.d);
      add_row<T>(xk, __shfl(dw, j), query_row(a, p, (uint32_t)(q0 + j)), a.d);
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t e = lane + 64u * i;
    if (e >= a.d) continue;
    if constexpr (SPLIT) {
      a.part_k[(part + row) * a.d + e] = xk[i] * a.scale;
      a.part_v[(part + row) * a.d + e] = xv[i];
    } else {
      a.dk[row * a.d + e] = (uint16_t)T::bits(xk[i] * a.scale);
      a.dv[row * a.d + e] = (uint16_t)T::bits(xv[i]);
    }
  }
}

// Fragments of its keys that a wave holds in registers; for heads of 128 all would be one more than
// there are registers for, and a spilled one waits for all loads in flight, the next
// tile's among them: the lane's own slot in LDS does not (8192 tokens, 64/8 heads of 128: 2310 us
// with one spilled, 2118 with three in LDS, which is what two workgroups a CU leave room for).
template <int DB>
constexpr int dkv_held() { return DB == 4 ? 5 : 2 * DB; }

template <int DB, bool ROW>
constexpr uint32_t dkv_buffer() { return 2u * tile_bytes<DB>() + (ROW ? 3u : 2u) * kAttnTile * 4u; }

// A workgroup of W waves takes 32 W keys, a wave 32 of them, keeps them and their values
// in registers and streams the queries that attend them, of all heads that share them,
// and their rows of dout past them in tiles of 64, so that the sums over queries and over
// heads are one, in a fixed order.  Per block of 32 queries: S = Q K^T, dP = dout V^T, p and
// dS as for dq; then dv^T += dout^T p and dk^T += Q^T dS.  p and dS are rounded to 16 bits (off
// by half a step of their own size, which the sums average out).  Bound by the matrix cores,
// 1050 TFLOP/s of the four products at that size, and by waits between two waves a SIMD.
//
// SPLIT: the queries in a.splits parts, each leaving fp32 sums.
template <class T, int DB, int W, bool ROW, bool SPLIT>
__global__ void __launch_bounds__(64 * W, 2) attn_dkv_kernel(const AttnArgs a) {
  extern __shared__ __align__(16) unsigned char lds[];
  __shared__ uint32_t found;  // an infinity or NaN among the queries or rows of dout of a tile that a mask cuts
  constexpr uint32_t kBytes = tile_bytes<DB>();
  constexpr uint32_t kBuf = dkv_buffer<DB, ROW>();  // queries, dout, l2, delta, and with rows tokens
  constexpr int kHeld = dkv_held<DB>();
  const uint32_t unit = SPLIT ? blockIdx.x / a.splits : blockIdx.x, split = SPLIT ? blockIdx.x % a.splits : 0u;
  const Place32 p = place_of<true>(a, unit, 32u * W);
  Lane ln;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63u, half = lane >> 5;
  const int32_t wg0 = (int32_t)(p.tile * (32u * W)), key0 = wg0 + (int32_t)wave * 32;
  if (p.live && wg0 < p.lk) {
    const int32_t key = key0 + (int32_t)(lane & 31u), at_key = min(key, p.lk - 1), R = p.lq * (int32_t)a.G;
    typename T::frag k[2 * DB], v[2 * DB];
    load_row<T, DB>(key_rows(a, p) + (uint64_t)at_key * a.k_row, key < p.lk, a.d, k);
    load_row<T, DB>(value_rows(a, p) + (uint64_t)at_key * a.v_row, key < p.lk, a.d, v);
    // rows [first, last) of the queries attend key x
    const auto first_row = [&](int32_t x) SDC_INLINE {
      return a.causal ? (int32_t)min((int64_t)max(x - (p.lk - p.lq), 0) * a.G, (int64_t)R) : 0;
    };
    const auto last_row = [&](int32_t x) SDC_INLINE {
      return a.window ? (int32_t)max(min(((int64_t)x - (p.lk - p.lq) + a.window) * a.G, (int64_t)R), (int64_t)0) : R;
    };
    // the lane's key is attended by rows [lo, lo + span)
    const int32_t lo = first_row(at_key);
    const uint32_t span = (uint32_t)max((key < p.lk ? last_row(at_key) : 0) - lo, 0);
    const int32_t wg_last = min(wg0 + 32 * W - 1, p.lk - 1), w_last = min(key0 + 31, p.lk - 1);
    const int32_t wg_begin = first_row(wg0), wg_end = last_row(wg_last);
    const bool idle = key0 >= p.lk;
    const int32_t begin = first_row(min(key0, p.lk - 1)), end = idle ? 0 : last_row(w_last);
    const int32_t from = first_row(w_last), to = key0 + 31 < p.lk ? last_row(key0) : 0;  // all of the wave's keys
    int32_t t0 = wg_begin / (int32_t)kAttnTile, t1 = max((wg_end + (int32_t)kAttnTile - 1) / (int32_t)kAttnTile, t0);
    if constexpr (SPLIT) {
      const int32_t each = (t1 - t0 + (int32_t)a.splits - 1) / (int32_t)a.splits;
      t0 = min(t0 + (int32_t)split * each, t1);
      t1 = min(t0 + each, t1);
    }
    const int shift = grad_shift<T>(a);
    const float f = power_of_two(shift - (int)kPShift<T>);
    f32x16 dk[DB], dv[DB];
#pragma unroll
    for (int m = 0; m < DB; ++m)
#pragma unroll
      for (int e = 0; e < 16; ++e) dk[m][e] = dv[m][e] = 0.0f;
    QueryLoader<DB, W> lq;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(SDC_LDS unsigned char*)lds;
    TileReads<T> at(lds0);
    const float *l2 = a.l2 + grouped_row(a, p, 0), *delta = a.delta + grouped_row(a, p, 0);
    const auto fill = [&](int32_t t, uint32_t buf) SDC_INLINE {
      const uint32_t r = (uint32_t)t * kAttnTile, base = lds0 + buf * kBuf;
      lq.fill(a, p, r, (uint32_t)R, base, base + kBytes);
      const uint32_t row = min(r + lane, (uint32_t)R - 1u);
      if (wave == 0) load4_to_lds(l2 + row, base + 2u * kBytes);
      if (wave == W - 1) load4_to_lds(delta + row, base + 2u * kBytes + 4u * kAttnTile);
      if (ROW && wave == 1)  // the rows' tokens, from the first's
        *(SDC_LDS uint32_t*)(uintptr_t)(base + 2u * kBytes + 8u * kAttnTile + 4u * lane) =
            token_of(a, r + lane) - token_of(a, r);
    };
    const uint32_t put = lds0 + 2u * kBuf + threadIdx.x * 16u;  // the lane's fragments of its key that LDS holds
#pragma unroll
    for (int i = kHeld; i < 2 * DB; ++i)
      *(SDC_LDS typename T::frag*)(uintptr_t)(put + (i - kHeld) * 16u * 64u * W) = k[i];
    if (t0 < t1) fill(t0, 0);
    // cut by a mask for some key of the workgroup
    const int32_t wg_from = first_row(wg_last), wg_to = wg0 + 32 * W <= p.lk ? last_row(wg0) : 0;
    if (threadIdx.x == 0) found = 0;
    uint32_t buf = 0;
    for (int32_t t = t0; t < t1; ++t, at.move(buf ? 0u - kBuf : kBuf), buf ^= 1u) {
      tile_barrier();  // this buffer is whole, and everyone has left the other
      if (t + 1 < t1) fill(t + 1, buf ^ 1u);
      const int32_t q0 = t * (int32_t)kAttnTile;
      const unsigned char *qt = lds + buf * kBuf, *dt = qt + kBytes;
      if (q0 < wg_from || q0 + (int32_t)kAttnTile > wg_to) {
        find_nonfinite<T, DB, W>(qt, &found);
        find_nonfinite<T, DB, W>(dt, &found);
      }
      if (q0 >= end || q0 + (int32_t)kAttnTile <= begin) continue;
      const bool masked = q0 < from || q0 + (int32_t)kAttnTile > to;
      const float *lt = reinterpret_cast<const float*>(dt + kBytes), *et = lt + kAttnTile;
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        f32x16 s, dp;
#pragma unroll
        for (int e = 0; e < 16; ++e) s[e] = dp[e] = 0.0f;
        // with rows the scores first, all that the row takes of them next: both products and the
        // row's sums at a time would not fit the registers
        const auto key_frag = [&](int i) SDC_INLINE {
          return i < kHeld ? k[i]
                           : *(const SDC_LDS typename T::frag*)(uintptr_t)(put + (i - kHeld) * 16u * 64u * W);
        };
#pragma unroll
        for (int i = 0; i < 2 * DB; ++i) {
          s = mfma32(at.row(0, n, i), key_frag(i), s);
          if constexpr (!ROW) dp = mfma32(at.row(kBytes, n, i), v[i], dp);
        }
        uint32_t first = (uint32_t)(q0 + 32 * n + 4 * (int32_t)half - lo);
        if constexpr (ROW) {
          // row r = token G + head of the queries is row token hq + head of the scores', so
          // token (hq - G) + r: the sums weighted by r and, where heads are grouped, by token
          if (masked) {
#pragma unroll
            for (int e = 0; e < 16; ++e) s[e] = first + element_row(e, 0) < span ? s[e] : 0.0f;
          }
          if (key < p.lk) {
            ScoreSums c;
            add_scores(c, s, 0);
            const uint32_t row = (uint32_t)q0 + 32u * n + 4u * half;
            const uint64_t at_row = (uint64_t)p.q0 * a.hq + p.head * a.G + row;
            join_scores(ln, c, at_row * a.kw + (uint32_t)key + 1u, a.kw);
            if (a.hq != a.G) {
              const uint32_t token = token_of(a, a.G != 1 ? (uint32_t)q0 : row);
              uint32_t tlo = c.wlo, thi = c.whi;
              if (a.G != 1) {
                tlo = thi = 0;
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                  const u32x4 w = *reinterpret_cast<const u32x4*>(et + kAttnTile + 32 * n + 8 * g + 4 * half);
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    const uint32_t x = __float_as_uint(s[4 * g + e]);
                    tlo = udot2(x, w[e], tlo);
                    thi = udot2(x, w[e] << 16, thi);
                  }
                }
              }
              ln.w += (uint64_t)(a.hq - a.G) * a.kw *
                      ((uint64_t)token * (c.lo + ((uint64_t)c.hi << 16)) + tlo + ((uint64_t)thi << 16));
            }
            if (c.odd != c.odd) ln.nf += nonfinite_scores(s);
          }
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int i = 0; i < 2 * DB; ++i) dp = mfma32(at.row(kBytes, n, i), v[i], dp);
        }
        f32x16 ds;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const f32x4 lse = *reinterpret_cast<const f32x4*>(lt + 32 * n + 8 * g + 4 * half);
          const f32x4 del = *reinterpret_cast<const f32x4*>(et + 32 * n + 8 * g + 4 * half);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float pr = __builtin_amdgcn_exp2f(__builtin_fmaf(s[4 * g + e], a.c, -lse[e]));
            s[4 * g + e] = pr;
            ds[4 * g + e] = pr * (dp[4 * g + e] - del[e]);
            if constexpr (kPShift<T> != 0.0f) ds[4 * g + e] *= f;
          }
        }
        if (masked) {
          asm volatile("" : "+v"(first));  // so that this stays a branch: no selects for the other tiles
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (first + element_row(e, 0) >= span) s[e] = ds[e] = 0.0f;
        }
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const typename T::frag w = operand<T>(s, i), x = operand<T>(ds, i);
#pragma unroll
          for (int m = 0; m < DB; ++m) {
            dv[m] = mfma32(at.column(kBytes, m, 2 * n + i), w, dv[m]);
            dk[m] = mfma32(at.column(0, m, 2 * n + i), x, dk[m]);
          }
        }
        __builtin_amdgcn_s_setprio(0);
      }
    }
    const uint64_t key_row = (uint64_t)(p.k0 + (uint32_t)key) * a.hk + p.head;
    const uint64_t all_rows = (uint64_t)(a.seq_k ? a.len_k : a.batch * a.len_k) * a.hk;
    __syncthreads();  // found is
    if (found) {
      for (int32_t x = key0; x < min(key0 + 32, p.lk); ++x)
        dkv_row<T, SPLIT>(a, p, x, max(first_row(x), t0 * (int32_t)kAttnTile),
                          min(last_row(x), t1 * (int32_t)kAttnTile), (uint64_t)(p.k0 + (uint32_t)x) * a.hk + p.head,
                          split * all_rows);
    } else if (key < p.lk) {
      const float gk = a.scale * power_of_two(-shift), gv = power_of_two(-(int)kPShift<T>);
#pragma unroll
      for (int m = 0; m < DB; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t x = 32u * m + 8u * e + 4u * half;
          if (x >= a.d) continue;
          const f32x4 xk = {dk[m][4 * e] * gk, dk[m][4 * e + 1] * gk, dk[m][4 * e + 2] * gk, dk[m][4 * e + 3] * gk};
          const f32x4 xv = {dv[m][4 * e] * gv, dv[m][4 * e + 1] * gv, dv[m][4 * e + 2] * gv, dv[m][4 * e + 3] * gv};
          if constexpr (SPLIT) {
            const uint64_t to_part = (split * all_rows + key_row) * a.d + x;
            *reinterpret_cast<f32x4*>(a.part_k + to_part) = xk;
            *reinterpret_cast<f32x4*>(a.part_v + to_part) = xv;
          } else {
            store4<T>(a.dk + key_row * a.d + x, xk.x, xk.y, xk.z, xk.w);
            store4<T>(a.dv + key_row * a.d + x, xv.x, xv.y, xv.z, xv.w);
          }
        }
    }
  }
  if constexpr (ROW) store_tile_row<W>(ln, a.rows + blockIdx.x);
}

// dk and dv: the splits' sums, in split order.  Eight elements a thread; rows outside every
// sequence have none.
template <class T>
__global__ void __launch_bounds__(256) attn_dkv_finish_kernel(const AttnArgs a, uint64_t rows) {
  const uint64_t all = rows * a.hk * a.d, at = ((uint64_t)blockIdx.x * 256u + threadIdx.x) * 8u;
  if (at >= all) return;
  if (a.seq_k) {
    const uint32_t row = (uint32_t)(at / ((uint64_t)a.hk * a.d));
    if (!in_sequences(a.seq_k, a.batch, a.len_k, row)) return;
  }
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    const float* part = (v ? a.part_v : a.part_k) + at;
    f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f}, y = x;
    for (uint32_t k = 0; k < a.splits; ++k) {
      x += *reinterpret_cast<const f32x4*>(part + k * all);
      y += *reinterpret_cast<const f32x4*>(part + k * all + 4);
    }
    uint16_t* out = (v ? a.dv : a.dk) + at;
    store4<T>(out, x.x, x.y, x.z, x.w);
    store4<T>(out + 4, y.x, y.y, y.z, y.w);
  }
}

}  // namespace

int32_t launch_attn_dkv(const AttnLaunch& l, const AttnArgs& a, hipStream_t s) {
  return for_dtype(l.dtype, [&](auto type) {
    typedef decltype(type) T;
    const auto shape = [&](auto db) {
      constexpr int DB = decltype(db)::value, W = 4;
      const dim3 grid(a.units * a.splits), block(64 * W);
      const uint32_t bytes =
          2u * (a.rows ? dkv_buffer<DB, true>() : dkv_buffer<DB, false>()) + (2 * DB - dkv_held<DB>()) * 1024u * W;
      const bool split = a.splits > 1;
      if (a.rows && split) hipLaunchKernelGGL((attn_dkv_kernel<T, DB, W, true, true>), grid, block, bytes, s, a);
      else if (a.rows) hipLaunchKernelGGL((attn_dkv_kernel<T, DB, W, true, false>), grid, block, bytes, s, a);
      else if (split) hipLaunchKernelGGL((attn_dkv_kernel<T, DB, W, false, true>), grid, block, bytes, s, a);
      else hipLaunchKernelGGL((attn_dkv_kernel<T, DB, W, false, false>), grid, block, bytes, s, a);
      return launch_status();
    };
    int32_t st = a.d <= 64   ? shape(std::integral_constant<int, 2>())
                 : a.d <= 96 ? shape(std::integral_constant<int, 3>())
                             : shape(std::integral_constant<int, 4>());
    if (st || a.splits == 1) return st;
    const uint64_t rows = a.seq_k ? a.len_k : (uint64_t)a.batch * a.len_k;
    hipLaunchKernelGGL(attn_dkv_finish_kernel<T>, dim3((uint32_t)((rows * a.hk * a.d / 8 + 255) / 256)), dim3(256), 0, s,
                       a, rows);
    return launch_status();
  });
}

}  // namespace sdc
