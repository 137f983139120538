// attn.hip -- softmax attention and its gradient, which computes the scores again,
// for gfx950.
//
//   s = q k^T   z = scale s over the pairs that attend   lse = log sum exp z
//   out = exp(z - lse) v
//   delta = sum dout out   p = exp(z - lse)   dp = dout v^T   dz = p (dp - delta)
//   dv = p^T dout   dq = scale dz k   dk = scale dz^T q
//
// The scores never reach memory; the gradient's recomputation of them is the one of
// AEGIS' check (review page, section "core method", item 4), and both passes can
// fingerprint them while they are in registers.  Nothing is added by atomics, so a
// replay's gradients have the same bits (AWS Machine Learning Blog, "Detecting and
// recovering from silent data corruption on Amazon SageMaker HyperPod", section "Check
// 2"): dq and (dk, dv) are two launches that each compute the scores, 7 products where
// one launch with atomics takes 5.
//
// Forward: one launch (csrc/attn_fwd.hip), with few queries the keys in splits that a
// second one joins.  Gradient: one that takes delta and lse in the order the others read
// them, then dk and dv (csrc/attn_dkv.hip), dq (csrc/attn_dq.hip).  Bound by the matrix
// cores and, beside them, LDS reads and the vector units' exponentials; few queries by
// reading keys and values.
#include "attn_device.h"

namespace sdc {
namespace {

// l2 and delta of every query, and for fp16 the largest sums of squares of the rows of
// dout and v (of finite ones, in sequences: others have no say in what fp16 can hold).  16
// lanes a row; bound by reading dout and out (8192 tokens, 64 heads of 128: 268 MB in
// 44 us, right after the passes that wrote them).
template <class T>
__global__ void __launch_bounds__(256) attn_delta_kernel(const AttnArgs a, const uint16_t* __restrict__ out,
                                                         const float* __restrict__ lse, uint64_t rows_q,
                                                         uint64_t rows_k, float* __restrict__ l2,
                                                         float* __restrict__ delta, float* __restrict__ norms) {
  constexpr bool kNorms = kPShift<T> != 0.0f;
  const uint32_t part = threadIdx.x & 15u, first = blockIdx.x * 16u + (threadIdx.x >> 4), step = gridDim.x * 16u;
  const uint16_t* dout = reinterpret_cast<const uint16_t*>(a.dout);
  float most = 0.0f;
  for (uint64_t n = first; n < rows_q * a.hq; n += step) {
    float s = 0.0f, sq = 0.0f;
    if (part * 8u < a.d) {
      const u32x4 x = *reinterpret_cast<const u32x4*>(dout + n * a.d + part * 8u);
      const u32x4 y = *reinterpret_cast<const u32x4*>(out + n * a.d + part * 8u);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float u = T::value(x[i] >> (16 * h) & 0xFFFFu), v = T::value(y[i] >> (16 * h) & 0xFFFFu);
          s += u * v;
          sq += u * u;
        }
    }
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) {
      s += __shfl_xor(s, off);
      if constexpr (kNorms) sq += __shfl_xor(sq, off);
    }
    const uint32_t row = (uint32_t)(n / a.hq), head = (uint32_t)(n % a.hq);
    if (part == 0) {
      const uint64_t at = ((uint64_t)(head / a.G) * rows_q + row) * a.G + head % a.G;
      const float x = lse[n];
      delta[at] = s;
      // a query that attends nothing has no probabilities
      l2[at] = x == -__builtin_inff() ? __builtin_inff() : x * kLog2e - kPShift<T>;
    }
    if constexpr (kNorms)
      if (sq < __builtin_inff() && (!a.seq_q || in_sequences(a.seq_q, a.batch, a.len_q, row)))
        most = __builtin_fmaxf(most, sq);
  }
  if constexpr (kNorms) {
    float most_v = 0.0f;
    for (uint64_t n = first; n < rows_k * a.hk; n += step) {
      const uint32_t row = (uint32_t)(n / a.hk), head = (uint32_t)(n % a.hk);
      const unsigned char* v = a.v + head * a.v_head;
      if (a.seq_k) v += (uint64_t)row * a.v_row;
      else v += (uint64_t)(row / a.len_k) * a.v_batch + (uint64_t)(row % a.len_k) * a.v_row;
      float sq = 0.0f;
      if (part * 8u < a.d) {
        const u32x4 x = *reinterpret_cast<const u32x4*>(v + part * 16u);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float u = T::value(x[i] & 0xFFFFu), w = T::value(x[i] >> 16);
          sq += u * u + w * w;
        }
      }
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) sq += __shfl_xor(sq, off);
      if (sq < __builtin_inff() && (!a.seq_k || in_sequences(a.seq_k, a.batch, a.len_k, row)))
        most_v = __builtin_fmaxf(most_v, sq);
    }
    __shared__ float waves[2][4];
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
      most = __builtin_fmaxf(most, __shfl_xor(most, off));
      most_v = __builtin_fmaxf(most_v, __shfl_xor(most_v, off));
    }
    if ((threadIdx.x & 63u) == 0) {
      waves[0][threadIdx.x >> 6] = most;
      waves[1][threadIdx.x >> 6] = most_v;
    }
    __syncthreads();
    if (threadIdx.x < 2) {
      float m = waves[threadIdx.x][0];
#pragma unroll
      for (int i = 1; i < 4; ++i) m = __builtin_fmaxf(m, waves[threadIdx.x][i]);
      norms[threadIdx.x * kNormParts + blockIdx.x] = m;
    }
  }
}

// ---- host ----------------------------------------------------------------------------
constexpr uint32_t kMaxUnits = 1u << 23;  // a grid has fewer than 2^32 threads

struct Attn {
  uint64_t rows_q, rows_k;
  uint32_t waves;                       // of the forward pass' and dq's workgroups
  uint32_t tiles_q, units_q, splits;    // splits: of the forward pass' keys
  uint32_t tiles_k, units_k, splits_k;  // of dk and dv: splits of the queries
};

int32_t check_attn(const sdc_attn* h) {
  if (h == nullptr) return SDC_ERR_INVALID;
  if (h->dtype != SDC_BF16 && h->dtype != SDC_F16) return SDC_ERR_DTYPE;
  if (h->flags != 0 || h->causal > 1 || h->d == 0 || h->heads_k == 0 || h->heads_q == 0 ||
      h->heads_q % h->heads_k != 0 || (h->window != 0 && !h->causal) || !(h->scale >= 0x1p-64f && h->scale <= 0x1p64f) ||
      (h->seq_q == nullptr) != (h->seq_k == nullptr))
    return SDC_ERR_INVALID;
  if (h->d % 8 != 0 || h->d > 128) return SDC_ERR_RANGE;
  if (h->batch >= 1ull << 24 || h->heads_q >= 1ull << 20 || h->len_q >= 1ull << 31 || h->len_k >= 1ull << 31)
    return SDC_ERR_RANGE;
  const bool packed = h->seq_q != nullptr;
  const uint64_t n = packed ? 1 : h->batch;
  if (n != 0 && (h->len_q > (1ull << 31) / n || h->len_k > (1ull << 31) / n)) return SDC_ERR_RANGE;
  const uint64_t rows_q = n * h->len_q, rows_k = n * h->len_k;
  if (rows_q * h->heads_q >= 1ull << 31 || rows_k * h->heads_k >= 1ull << 31) return SDC_ERR_RANGE;
  if ((rows_q > 0 && h->q == nullptr) || (rows_k > 0 && (h->k == nullptr || h->v == nullptr))) return SDC_ERR_INVALID;
  const struct {
    const void* p;
    const uint64_t* stride;
    uint64_t rows, heads;
  } each[3] = {{h->q, h->q_stride, h->len_q, h->heads_q},
               {h->k, h->k_stride, h->len_k, h->heads_k},
               {h->v, h->v_stride, h->len_k, h->heads_k}};
  for (const auto& t : each) {
    if (reinterpret_cast<uintptr_t>(t.p) % 16 || (n > 1 && t.stride[0] % 8) || (t.rows > 1 && t.stride[1] % 8) ||
        (t.heads > 1 && t.stride[2] % 8))
      return SDC_ERR_ALIGN;
    if ((n > 1 && t.stride[0] >= 1ull << 40) || (t.rows > 1 && t.stride[1] >= 1ull << 23) ||
        (t.heads > 1 && t.stride[2] >= 1ull << 40))
      return SDC_ERR_RANGE;
  }
  if (reinterpret_cast<uintptr_t>(h->seq_q) % 4 || reinterpret_cast<uintptr_t>(h->seq_k) % 4) return SDC_ERR_ALIGN;
  // one tile of 32 queries, or of 128 keys, for each row at least
  if (rows_q * h->heads_q / 32 + h->batch * h->heads_k * 2 >= kMaxUnits ||
      rows_k * h->heads_k / 128 + h->batch * h->heads_k * 2 >= kMaxUnits)
    return SDC_ERR_RANGE;
  return SDC_OK;
}

Attn plan_attn(const sdc_attn* h) {
  Attn p;
  const bool packed = h->seq_q != nullptr;
  const uint64_t n = packed ? 1 : h->batch, G = h->heads_q / h->heads_k;
  p.rows_q = n * h->len_q;
  p.rows_k = n * h->len_k;
  // of a sequence, on average
  const uint64_t some = std::max<uint64_t>(h->batch, 1);
  const uint64_t len_q = packed ? (h->len_q + some - 1) / some : h->len_q;
  const uint64_t len_k = packed ? (h->len_k + some - 1) / some : h->len_k;
  const uint64_t each = h->heads_k * (packed ? 1 : h->batch);
  // Enough workgroups to fill the chip, of at least four tiles of keys; at most 64 for a tile
  // of queries, which is what the launch that joins them takes.
  const auto with_waves = [&](uint32_t waves, uint32_t per_cu) {
    const uint32_t rows = 32 * waves;
    const uint64_t keys = h->window ? std::min<uint64_t>(len_k, h->window + rows / G + 1) : len_k;
    p.waves = waves;
    p.tiles_q = packed ? (uint32_t)(h->len_q * G / rows + h->batch) : tiles(h->len_q * G, rows);
    p.units_q = (uint32_t)(p.tiles_q * each);
    p.splits = (uint32_t)std::max<uint64_t>(
        1, std::min<uint64_t>({per_cu * kCus / std::max(p.units_q, 1u), tiles(keys, 4 * kAttnTile), 64}));
  };
  // Up to 32 rows of queries: workgroups of one wave, whose single buffer is 8 kB for each 32
  // elements of a row, as many of them as run on a CU at once.  8 sequences of 8191 keys, 32/8
  // heads, one query each, with 4 / 5 / 6 / 8 of them a CU: 62.6 / 71.1 / 67.5 / 66.3 us with
  // heads of 128, 48.6 / 50.9 / 45.9 / 49.2 of 80 and (8192 keys) 41.7 / 36.4 / 36.9 / 43.8 of
  // 64.  Where even the splits leave fewer than three of them a CU, four waves that share the
  // loads of a tile hide more of their latency: one sequence of 8191 keys 22.8 -> 21.5 us, of
  // 65536 keys 71.0 -> 66.4; but 128 sequences of 2048 keys take 206 us so, and 197 with one.
  if (len_q * G <= 32) with_waves(1, h->d > 96 ? 4 : 6);
  if (len_q * G > 32 || (uint64_t)p.units_q * p.splits < 3 * kCus) with_waves(4, 2);
  p.tiles_k = packed ? (uint32_t)(h->len_k / 128) + (uint32_t)h->batch : tiles(h->len_k, 128);
  p.units_k = (uint32_t)(p.tiles_k * each);
  uint64_t queries = len_q;
  if (h->window) queries = std::min<uint64_t>(queries, h->window + 128);
  // Key tiles: two workgroups a CU, and twice that, so that the short sums that a causal mask
  // leaves even out, where a split still has 64 tiles of queries: its fp32 sums are written
  // and read again.  Measured (dk and dv in us, one split / two; two / four): 8192 tokens, 64/8
  // heads of 128 3105 / 2068, 2 x 4096, 16/4 heads of 80 323 / 255, but 2 x 2048, 16 heads of 128 114 /
  // 126.
  const uint32_t tiles_of_q = tiles(queries * G, kAttnTile), units = std::max(p.units_k, 1u);
  p.splits_k = std::max(1u, std::min({4 * kCus / units, std::max(2 * kCus / units, tiles_of_q / 64), tiles_of_q / 8}));
  return p;
}

struct AttnLayout {
  uint64_t rows, part, ml, l2, delta, norms, part_k, part_v, end;
};

AttnLayout layout_attn(const sdc_attn* h, const Attn& p, bool grad) {
  AttnLayout o;
  uint64_t at = 0;
  const auto take = [&](uint64_t bytes) {
    const uint64_t here = at;
    at = up(at + bytes, 256);
    return here;
  };
  const uint64_t q = p.rows_q * h->heads_q, k = p.rows_k * h->heads_k;
  o.rows = take(32ull * (grad ? (uint64_t)p.units_q + (uint64_t)p.units_k * p.splits_k + 1
                              : (uint64_t)p.units_q * p.splits));
  o.part = take(!grad && p.splits > 1 ? 4ull * p.splits * q * h->d : 0);
  o.ml = take(!grad && p.splits > 1 ? 8ull * p.splits * q : 0);
  o.l2 = take(grad ? 4ull * q : 0);
  o.delta = take(grad ? 4ull * q : 0);
  o.norms = take(grad ? 8ull * kNormParts : 0);
  o.part_k = take(grad && p.splits_k > 1 ? 4ull * p.splits_k * k * h->d : 0);
  o.part_v = take(grad && p.splits_k > 1 ? 4ull * p.splits_k * k * h->d : 0);
  o.end = std::max<uint64_t>(at, 256);
  return o;
}

AttnArgs attn_args(const sdc_attn* h) {
  AttnArgs a = {};
  a.q = static_cast<const unsigned char*>(h->q);
  a.k = static_cast<const unsigned char*>(h->k);
  a.v = static_cast<const unsigned char*>(h->v);
  a.q_batch = 2 * h->q_stride[0];
  a.k_batch = 2 * h->k_stride[0];
  a.v_batch = 2 * h->v_stride[0];
  // of one row, whatever its stride says
  a.q_row = h->len_q > 1 ? (uint32_t)(2 * h->q_stride[1]) : 0u;
  a.k_row = h->len_k > 1 ? (uint32_t)(2 * h->k_stride[1]) : 0u;
  a.v_row = h->len_k > 1 ? (uint32_t)(2 * h->v_stride[1]) : 0u;
  a.q_head = h->heads_q > 1 ? 2 * h->q_stride[2] : 0;
  a.k_head = h->heads_k > 1 ? 2 * h->k_stride[2] : 0;
  a.v_head = h->heads_k > 1 ? 2 * h->v_stride[2] : 0;
  a.seq_q = h->seq_q;
  a.seq_k = h->seq_k;
  a.batch = (uint32_t)h->batch;
  a.len_q = (uint32_t)h->len_q;
  a.len_k = (uint32_t)h->len_k;
  a.hq = (uint32_t)h->heads_q;
  a.hk = (uint32_t)h->heads_k;
  a.G = a.hq / a.hk;
  a.d = (uint32_t)h->d;
  // r / G for r below 2^31: with 2^s >= G, m = floor(2^(31+s) / G) + 1 is below 2^32 and off by
  // less than 2^s in 2^(31+s), so r m / 2^(31+s) passes r / G by less than 1 / G
  uint32_t s = 0;
  while ((1ull << s) < a.G) ++s;
  a.g_mul = (uint32_t)((1ull << (31 + s)) / a.G + (a.G > 1 ? 1 : 0));
  a.g_shift = 31 + s;
  a.causal = h->causal;
  a.window = (uint32_t)std::min<uint64_t>(h->window, 0x7FFFFFFFu);
  a.scale = h->scale;
  a.c = h->scale * kLog2e;
  a.splits = 1;
  a.kw = h->len_k;
  return a;
}

}  // namespace
}  // namespace sdc

using namespace sdc;

extern "C" int32_t sdc_attention_ws_bytes(const sdc_attn* h, uint64_t* h_bytes, uint64_t* h_grad_bytes) {
  int32_t st = check_attn(h);
  if (st) return st;
  const Attn p = plan_attn(h);
  if (h_bytes) *h_bytes = layout_attn(h, p, false).end;
  if (h_grad_bytes) *h_grad_bytes = layout_attn(h, p, true).end;
  return SDC_OK;
}

extern "C" int32_t sdc_attention(const sdc_attn* h, void* d_ws, uint64_t ws_bytes, void* d_out, float* d_lse,
                                 sdc_row* d_row, sdc_stream_t stream) {
  int32_t st = check_attn(h);
  if (st) return st;
  const Attn p = plan_attn(h);
  if (d_ws == nullptr || (p.rows_q > 0 && (d_out == nullptr || d_lse == nullptr))) return SDC_ERR_INVALID;
  if (reinterpret_cast<uintptr_t>(d_ws) % 16 || reinterpret_cast<uintptr_t>(d_row) % 16 ||
      reinterpret_cast<uintptr_t>(d_out) % 16 || reinterpret_cast<uintptr_t>(d_lse) % 4)
    return SDC_ERR_ALIGN;
  const AttnLayout o = layout_attn(h, p, false);
  if (ws_bytes < o.end) return SDC_ERR_WORKSPACE;
  hipStream_t s = as_stream(stream);
  unsigned char* ws = static_cast<unsigned char*>(d_ws);
  sdc_row* rows = reinterpret_cast<sdc_row*>(ws + o.rows);
  if (p.units_q > 0) {
    AttnArgs a = attn_args(h);
    a.tiles = p.tiles_q;
    a.units = p.units_q;
    a.splits = p.splits;
    a.rows = d_row ? rows : nullptr;
    a.out = static_cast<uint16_t*>(d_out);
    a.lse = d_lse;
    a.part = reinterpret_cast<float*>(ws + o.part);
    a.part_ml = reinterpret_cast<float2*>(ws + o.ml);
    if ((st = launch_attn(AttnLaunch{h->dtype, p.waves}, a, s))) return st;
  }
  return d_row ? launch_merge_tile_rows(rows, p.units_q * p.splits, nullptr, 0, d_row, nullptr, s) : SDC_OK;
}

extern "C" int32_t sdc_attention_grad(const sdc_attn* h, const void* d_out, const float* d_lse, const void* d_dout,
                                      void* d_ws, uint64_t ws_bytes, void* d_dq, void* d_dk, void* d_dv,
                                      const sdc_row* d_ref, uint32_t col_mask, sdc_row* d_row, uint32_t* d_mismatch,
                                      sdc_stream_t stream) {
  int32_t st = check_attn(h);
  if (st) return st;
  const Attn p = plan_attn(h);
  if (d_ws == nullptr || (d_dk == nullptr) != (d_dv == nullptr) ||
      (p.rows_q > 0 && p.rows_k > 0 && d_dq == nullptr && d_dk == nullptr) ||
      (p.rows_q > 0 && (d_out == nullptr || d_lse == nullptr || d_dout == nullptr)))
    return SDC_ERR_INVALID;
  if (d_ref != nullptr && (d_row == nullptr || d_mismatch == nullptr || col_mask == 0 || (col_mask & ~15u)))
    return SDC_ERR_INVALID;
  for (const void* x : {d_out, d_dout, (const void*)d_ws, (const void*)d_dq, (const void*)d_dk, (const void*)d_dv,
                        (const void*)d_ref, (const void*)d_row})
    if (reinterpret_cast<uintptr_t>(x) % 16) return SDC_ERR_ALIGN;
  if (reinterpret_cast<uintptr_t>(d_lse) % 4 || reinterpret_cast<uintptr_t>(d_mismatch) % 4) return SDC_ERR_ALIGN;
  const AttnLayout o = layout_attn(h, p, true);
  if (ws_bytes < o.end) return SDC_ERR_WORKSPACE;
  hipStream_t s = as_stream(stream);
  unsigned char* ws = static_cast<unsigned char*>(d_ws);
  sdc_row *rows_q = reinterpret_cast<sdc_row*>(ws + o.rows), *rows_k = rows_q + p.units_q;
  const uint32_t n_rows_k = p.units_k * p.splits_k;
  AttnArgs a = attn_args(h);
  a.dout = static_cast<const unsigned char*>(d_dout);
  float *l2 = reinterpret_cast<float*>(ws + o.l2), *delta = reinterpret_cast<float*>(ws + o.delta);
  float* norms = reinterpret_cast<float*>(ws + o.norms);
  if (p.rows_q > 0) {
    // fp16 takes all parts of the norms
    const uint64_t n = (p.rows_q * h->heads_q + 15) / 16;
    const dim3 grid(h->dtype == SDC_F16 ? kNormParts : (uint32_t)std::min<uint64_t>(n, 8 * kCus));
    st = for_dtype(h->dtype, [&](auto t) {
      hipLaunchKernelGGL(attn_delta_kernel<decltype(t)>, grid, dim3(256), 0, s, a,
                         static_cast<const uint16_t*>(d_out), d_lse, p.rows_q, p.rows_k, l2, delta, norms);
      return launch_status();
    });
    if (st) return st;
  }
  a.l2 = l2;
  a.delta = delta;
  a.norms = norms;
  const bool keys = d_dk != nullptr && p.units_k > 0, queries = d_dq != nullptr && p.units_q > 0;
  if (keys) {
    a.tiles = p.tiles_k;
    a.units = p.units_k;
    a.splits = p.splits_k;
    a.rows = d_row ? rows_k : nullptr;
    a.dk = static_cast<uint16_t*>(d_dk);
    a.dv = static_cast<uint16_t*>(d_dv);
    a.part_k = reinterpret_cast<float*>(ws + o.part_k);
    a.part_v = reinterpret_cast<float*>(ws + o.part_v);
    if ((st = launch_attn_dkv(AttnLaunch{h->dtype, 4}, a, s))) return st;
  }
  if (queries) {
    a.tiles = p.tiles_q;
    a.units = p.units_q;
    a.splits = 1;
    a.rows = d_row ? rows_q : nullptr;
    a.dq = static_cast<uint16_t*>(d_dq);
    if ((st = launch_attn_dq(AttnLaunch{h->dtype, p.waves}, a, s))) return st;
  }
  if (!d_row) return SDC_OK;
  // both launches compute the scores; d_row is dk's and dv's where those ran
  if (queries && keys &&
      (st = launch_merge_tile_rows(rows_q, p.units_q, d_ref, col_mask, rows_k + n_rows_k, d_mismatch, s)))
    return st;
  return keys ? launch_merge_tile_rows(rows_k, n_rows_k, d_ref, col_mask, d_row, d_mismatch, s)
              : launch_merge_tile_rows(rows_q, queries ? p.units_q : 0, d_ref, col_mask, d_row, d_mismatch, s);
}
