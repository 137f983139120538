// attn_device.h -- the tiled kernels of softmax attention (csrc/attn.hip says what
// they compute) and what they share.
//
// Rows and columns.  The queries of the G heads that share a head of keys are one
// matrix of lq G rows, r = token G + head, so a tile of keys in LDS serves all of them
// and a few tokens of many heads still fill a tile.  Products are 32 x 32 x 16 MFMA of
// 16-bit operands into fp32:
//   forward, dq   S^T = K Q^T: keys down, queries across.  A lane holds 16 of a
//                 query's 32 keys (the lane 32 further on the other 16), so a query's
//                 maximum and sum are in-lane but for one exchange of halves.
//   dk, dv        S = Q K^T: queries down, keys across.
// The result of such a product has, in lane (column, half), element r of row
//   8 (r >> 2) + 4 half + (r & 3);
// as the right operand of the next product, whose sum runs over those rows, a lane
// has to give 8 rows of every 16, and the sum's order is free as long as the left
// operand has the same: so a lane's elements 0 .. 7 and 8 .. 15, converted, are the
// two operands, without an exchange, and the left operand is read transposed from
// LDS in that order (two reads of four rows of a column each).
//
// LDS holds a tile of 64 rows in groups of 32 elements: 64 pieces of 64 bytes, as direct
// loads write them (16 rows a load), whose four 16-byte chunks are permuted by an exclusive or
// with (row >> 2) & 3.  Both kinds of reads, a chunk of 16 rows and, transposed, four chunks of 8
// rows, then fall on all banks alike, and a read's address is one of two registers and a
// constant, whichever group, block or step it takes.
#pragma once

#include "tile_device.h"

namespace sdc {

struct AttnArgs {
  const unsigned char *q, *k, *v;
  uint64_t q_batch, k_batch, v_batch;  // bytes from one entry of the batch to the next
  uint64_t q_head, k_head, v_head;
  uint32_t q_row, k_row, v_row;
  const int32_t *seq_q, *seq_k;        // packed sequences' first rows, or null
  uint32_t batch, len_q, len_k;        // rows of an entry, or of all packed sequences
  uint32_t hq, hk, G, d;
  uint32_t g_mul, g_shift;             // r / G = r g_mul >> g_shift for r below 2^31
  uint32_t causal, window;             // window 0: none
  float scale, c;                      // c = scale log2(e)
  uint32_t tiles;                      // of an entry (packed: of all, at most)
  uint32_t units;                      // tiles x heads of keys (x entries)
  uint32_t splits;
  uint64_t kw;                         // columns of the scores that the fingerprint row describes
  sdc_row* rows;                       // one partial row per workgroup, or null
  uint16_t* out;
  float* lse;                          // [rows][hq]
  float* part;                         // splits: their sums, [hk][rows G][split][d]
  float2* part_ml;                     // and their reference exponents and sums of exponentials
  // gradient
  const unsigned char* dout;           // contiguous, as out
  const float *l2, *delta;             // [hk][rows G]: lse log2(e) (less kPShift), sum dout out
  const float* norms;                  // fp16: kNormParts largest sums of squares of rows of dout, and as many of v
  uint16_t *dq, *dk, *dv;
  float *part_k, *part_v;              // splits of the queries: [split][rows of keys][hk][d]
};

struct AttnLaunch {
  uint32_t dtype;
  uint32_t waves;  // of 32 queries (keys, for dk and dv)
};
int32_t launch_attn(const AttnLaunch& l, const AttnArgs& a, hipStream_t s);
int32_t launch_attn_dq(const AttnLaunch& l, const AttnArgs& a, hipStream_t s);
int32_t launch_attn_dkv(const AttnLaunch& l, const AttnArgs& a, hipStream_t s);

// Workgroups of the gradient's first launch, at most, and so parts of fp16's norms.
constexpr uint32_t kNormParts = 512;

// Rows (of keys; of queries for dk and dv) of a tile in LDS.
constexpr uint32_t kAttnTile = 64;

namespace {

// For lambdas that several places call.
#define SDC_INLINE __attribute__((always_inline))

typedef float f32x16 __attribute__((ext_vector_type(16)));

// fp16: probabilities are held 2^14 times as large (at most 2^14), out of the subnormals
template <class T> constexpr float kPShift = 0.0f;
template <> constexpr float kPShift<Fp16> = 14.0f;

__device__ __forceinline__ f32x16 mfma32(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mfma32(f16x8 a, f16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

// Row of element r of a 32 x 32 result in a lane of half `half`.
__device__ __forceinline__ constexpr uint32_t element_row(uint32_t r, uint32_t half) {
  return 8u * (r >> 2) + 4u * half + (r & 3u);
}

// x, which every lane of the wave has, in a scalar register.
__device__ __forceinline__ int32_t uniform(int32_t x) { return __builtin_amdgcn_readfirstlane(x); }

__device__ __forceinline__ const unsigned char* uniform(const unsigned char* p) {
  const uint64_t x = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = (uint32_t)uniform((int32_t)(uint32_t)x), hi = (uint32_t)uniform((int32_t)(uint32_t)(x >> 32));
  return reinterpret_cast<const unsigned char*>((uint64_t)hi << 32 | lo);
}

// A value and the one of the lane 32 further on (or back).
__device__ __forceinline__ float both_max(float x) {
  const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __builtin_fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
}
__device__ __forceinline__ float both_sum(float x) {
  const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}

// Elements 8 h .. 8 h + 7 of a result as an operand, rounded to nearest.
template <class T>
__device__ __forceinline__ typename T::frag operand(const f32x16& x, int h) {
  typedef float f32x8 __attribute__((ext_vector_type(8)));
  const f32x8 y = {x[8 * h], x[8 * h + 1], x[8 * h + 2], x[8 * h + 3], x[8 * h + 4], x[8 * h + 5], x[8 * h + 6], x[8 * h + 7]};
  return __builtin_convertvector(y, typename T::frag);
}

// ---- sequences -------------------------------------------------------------------

// The part of the batch that a workgroup works on.
struct Place32 {
  uint32_t seq, tile, head;
  uint32_t q0, k0;   // first rows in the batch
  int32_t lq, lk;
  bool live;
};

__device__ __forceinline__ uint32_t seq_at(const int32_t* s, uint32_t i, uint32_t rows) {
  const int32_t x = s[i];
  return x < 0 ? 0u : min((uint32_t)x, rows);
}

// Whether a row lies in one of the sequences, whose offsets ascend.
__device__ __forceinline__ bool in_sequences(const int32_t* s, uint32_t batch, uint32_t rows, uint32_t row) {
  return seq_at(s, 0, rows) <= row && row < seq_at(s, batch, rows);
}

// Unit -> sequence, tile, head of keys.  Heads run fastest, then sequences, and later
// tiles, which attend more keys under a causal mask, come first.  For packed sequences
// the tiles are counted from their offsets, 64 sequences at a time; there may be fewer
// than units.  KEYS: tiles of `rows` keys (the first come first), else of `rows` queries
// of G heads.
template <bool KEYS>
__device__ __forceinline__ Place32 place_of(const AttnArgs& a, uint32_t unit, uint32_t rows) {
  Place32 p;
  p.head = unit % a.hk;
  uint32_t j = unit / a.hk;
  p.live = true;
  if (!a.seq_q) {
    p.seq = j % a.batch;
    j /= a.batch;
    p.tile = KEYS ? j : a.tiles - 1u - j;
    p.q0 = p.seq * a.len_q;
    p.k0 = p.seq * a.len_k;
    p.lq = (int32_t)a.len_q;
    p.lk = (int32_t)a.len_k;
    return p;
  }
  const uint32_t lane = threadIdx.x & 63u;
  const int32_t* s = KEYS ? a.seq_k : a.seq_q;
  const uint32_t all = KEYS ? a.len_k : a.len_q, each = KEYS ? 1u : a.G;
  p.live = false;
  p.seq = p.tile = 0;
  for (uint32_t b = 0; b < a.batch; b += 64) {
    uint32_t n = 0;
    if (b + lane < a.batch) {
      const uint32_t lo = seq_at(s, b + lane, all), hi = seq_at(s, b + lane + 1u, all);
      n = hi > lo ? (uint32_t)(((uint64_t)(hi - lo) * each + rows - 1u) / rows) : 0u;
    }
    uint32_t sum = n;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const uint32_t x = __shfl_up(sum, off);
      if ((int)lane >= off) sum += x;
    }
    const uint64_t past = __ballot(sum > j);
    if (past) {
      const int at = __builtin_ctzll(past);
      const uint32_t end = __shfl(sum, at), mine = __shfl(n, at), i = j - (end - mine);
      p.seq = b + (uint32_t)at;
      p.tile = KEYS ? i : mine - 1u - i;
      p.live = true;
      break;
    }
    j -= __shfl(sum, 63);
  }
  p.seq = __builtin_amdgcn_readfirstlane(p.seq);
  p.tile = __builtin_amdgcn_readfirstlane(p.tile);
  const uint32_t q0 = seq_at(a.seq_q, p.seq, a.len_q), q1 = seq_at(a.seq_q, p.seq + 1u, a.len_q);
  const uint32_t k0 = seq_at(a.seq_k, p.seq, a.len_k), k1 = seq_at(a.seq_k, p.seq + 1u, a.len_k);
  p.q0 = __builtin_amdgcn_readfirstlane(q0);
  p.k0 = __builtin_amdgcn_readfirstlane(k0);
  p.lq = (int32_t)__builtin_amdgcn_readfirstlane(q1 > q0 ? q1 - q0 : 0u);
  p.lk = (int32_t)__builtin_amdgcn_readfirstlane(k1 > k0 ? k1 - k0 : 0u);
  return p;
}

__device__ __forceinline__ uint32_t token_of(const AttnArgs& a, uint32_t r) {
  return (uint32_t)(((uint64_t)r * a.g_mul) >> a.g_shift);
}

// Keys [lo, hi) that token t attends.
__device__ __forceinline__ int32_t keys_end(const AttnArgs& a, const Place32& p, int32_t t) {
  return a.causal ? min(t + 1 + p.lk - p.lq, p.lk) : p.lk;
}
__device__ __forceinline__ int32_t keys_begin(const AttnArgs& a, const Place32& p, int32_t t) {
  return a.window ? max((int32_t)max((int64_t)t + 1 + p.lk - p.lq - (int64_t)a.window, (int64_t)0), 0) : 0;
}

// Address of row r of the queries (or, contiguous, of dout and out) of a head of keys.
__device__ __forceinline__ const unsigned char* query_row(const AttnArgs& a, const Place32& p, uint32_t r) {
  const uint32_t t = token_of(a, r), g = r - t * a.G;
  const uint64_t row = a.seq_q ? (uint64_t)(p.q0 + t) : (uint64_t)t;
  return a.q + (a.seq_q ? 0u : p.seq * a.q_batch) + row * a.q_row + (uint64_t)(p.head * a.G + g) * a.q_head;
}
__device__ __forceinline__ uint64_t flat_row(const AttnArgs& a, const Place32& p, uint32_t r) {
  const uint32_t t = token_of(a, r), g = r - t * a.G;
  return (uint64_t)(p.q0 + t) * a.hq + p.head * a.G + g;  // of [rows][hq]
}
__device__ __forceinline__ uint64_t grouped_row(const AttnArgs& a, const Place32& p, uint32_t r) {
  const uint64_t all = (uint64_t)(a.seq_q ? a.len_q : a.batch * a.len_q) * a.G;
  return (uint64_t)p.head * all + (uint64_t)p.q0 * a.G + r;  // of [hk][rows G]
}
__device__ __forceinline__ const unsigned char* key_rows(const AttnArgs& a, const Place32& p) {
  return a.k + (a.seq_q ? (uint64_t)p.k0 * a.k_row : p.seq * a.k_batch) + p.head * a.k_head;
}
__device__ __forceinline__ const unsigned char* value_rows(const AttnArgs& a, const Place32& p) {
  return a.v + (a.seq_q ? (uint64_t)p.k0 * a.v_row : p.seq * a.v_batch) + p.head * a.v_head;
}

// ---- tiles in LDS ----------------------------------------------------------------

// 64 rows of up to 32 DB elements.
constexpr uint32_t kGroup = kAttnTile * 64u;  // bytes of 32 elements of each
template <int DB>
constexpr uint32_t tile_bytes() { return DB * kGroup; }
__device__ __forceinline__ uint32_t chunk_swizzle(uint32_t row) { return row >> 2 & 3u; }

// 16 bytes per lane from base + off to LDS at lds + 16 * lane (base, lds uniform); see load_to_lds.
__device__ __forceinline__ void load_to_lds_from(const unsigned char* base, uint32_t off, uint32_t lds) {
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %1, %2"
      :
      : "s"(lds), "v"(off), "s"(base)
      : "m0", "memory");
#pragma clang diagnostic pop
}

// 4 bytes per lane to LDS at lds + 4 * lane (lds uniform); see load_to_lds.
__device__ __forceinline__ void load4_to_lds(const float* src, uint32_t lds) {
  lds = (uint32_t)uniform((int32_t)lds);
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dword %1, off"
      :
      : "s"(lds), "v"(src)
      : "m0", "memory");
#pragma clang diagnostic pop
}

// Fills a tile with rows of a matrix, all waves together: what lies past its last row
// or past its width is zero, so that nothing there can reach a sum.
template <int DB, int WAVES>
struct TileLoader {
  static constexpr uint32_t kBlocks = 4 / WAVES;  // of 16 rows, of a wave
  static_assert(kBlocks * WAVES == 4, "the waves' rows cover a tile");
  const unsigned char* base;  // of the matrix' first row
  uint32_t stride, width;     // bytes
  uint32_t row, at, off;      // of the lane within 16 rows: row, byte of its chunk, both from base
  bool in;                    // whole groups

  __device__ __forceinline__ void init(const unsigned char* b, uint32_t row_bytes, uint32_t d) {
    const uint32_t lane = threadIdx.x & 63u;
    base = b;
    stride = row_bytes;
    width = 2u * d;
    row = lane >> 2;
    at = ((lane & 3u) ^ chunk_swizzle(row)) * 16u;
    off = row * stride + at;
    in = width == 64u * DB;
  }
  // Rows first .. first + 63, of `rows` rows, into LDS at byte `lds`.
  __device__ __forceinline__ void fill(uint32_t first, uint32_t rows, uint32_t lds) const {
    const uint32_t block = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * kBlocks;
    const bool whole = in && first + kAttnTile <= rows;
#pragma unroll
    for (uint32_t i = 0; i < kBlocks; ++i) {
      const uint32_t r = first + (block + i) * 16u, to = (uint32_t)uniform((int32_t)(lds + (block + i) * 1024u));
      const unsigned char* from = uniform(base + (uint64_t)r * stride);
      if (whole) {
#pragma unroll
        for (uint32_t m = 0; m < DB; ++m) load_to_lds_from(from + m * 64u, off, to + m * kGroup);
      } else {
        const unsigned char* zero = reinterpret_cast<const unsigned char*>(&g_zero16);
#pragma unroll
        for (uint32_t m = 0; m < DB; ++m)
          load_to_lds(r + row < rows && m * 64u + at < width ? from + m * 64u + off : zero, to + m * kGroup);
      }
    }
  }
};

// The queries' and dout's rows, whose places follow from token and head.
template <int DB, int WAVES>
struct QueryLoader {
  static_assert(WAVES == 4, "a wave has 16 rows of a tile");
  __device__ __forceinline__ void fill(const AttnArgs& a, const Place32& p, uint32_t first, uint32_t rows,
                                       uint32_t lds_q, uint32_t lds_do) const {
    lds_q = (uint32_t)uniform((int32_t)lds_q);
    lds_do = (uint32_t)uniform((int32_t)lds_do);
    const uint32_t lane = threadIdx.x & 63u, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t r = first + wave * 16u + (lane >> 2), at = ((lane & 3u) ^ chunk_swizzle(lane >> 2)) * 16u;
    const unsigned char* zero = reinterpret_cast<const unsigned char*>(&g_zero16);
    const unsigned char* q = query_row(a, p, min(r, rows - 1u)) + at;
    const unsigned char* o = a.dout + flat_row(a, p, min(r, rows - 1u)) * (2u * a.d) + at;
    const bool whole = a.d == 32u * DB && first + kAttnTile <= rows;
#pragma unroll
    for (uint32_t m = 0; m < DB; ++m) {
      const bool has = whole || (r < rows && m * 64u + at < 2u * a.d);
      load_to_lds(has ? q + m * 64u : zero, lds_q + wave * 1024u + m * kGroup);
      load_to_lds(has ? o + m * 64u : zero, lds_do + wave * 1024u + m * kGroup);
    }
  }
};

// A lane's reads of the tile at LDS byte `tile` as the left operand.
template <class T>
struct TileReads {
  uint32_t row0, row1, col0, col1;
  __device__ __forceinline__ explicit TileReads(uint32_t tile) {
    const uint32_t lane = threadIdx.x & 63u, half = lane >> 5;
    const uint32_t rows = (lane & 31u) * 64u + ((half ^ chunk_swizzle(lane & 31u)) << 4);
    const uint32_t r = 4u * half + (lane >> 2 & 3u), chunk = (lane >> 4 & 1u) * 2u + (lane >> 1 & 1u);
    const uint32_t cols = r * 64u + ((chunk ^ chunk_swizzle(r)) << 4) + (lane & 1u) * 8u;
    row0 = tile + rows;
    row1 = tile + (rows ^ 32u);
    col0 = tile + cols;
    col1 = tile + (cols ^ 32u) + 512u;  // eight rows on, the swizzle's bit 1 is the other one
  }
  // The same of the tile `by` bytes on.  (Kept as they are: a read's constant then fits its
  // instruction.)
  __device__ __forceinline__ void move_rows(uint32_t by) {
    row0 += by;
    row1 += by;
    asm volatile("" : "+v"(row0), "+v"(row1));
  }
  __device__ __forceinline__ void move_columns(uint32_t by) {
    col0 += by;
    col1 += by;
    asm volatile("" : "+v"(col0), "+v"(col1));
  }
  __device__ __forceinline__ void move(uint32_t by) {
    move_rows(by);
    move_columns(by);
  }
  // Rows 32 b .. of the tile, elements 16 s .. of each: the sum runs along the rows.
  // tile: bytes to another one, a constant.
  __device__ __forceinline__ typename T::frag row(uint32_t tile, int b, int s) const {
    return *(const SDC_LDS typename T::frag*)(uintptr_t)((s & 1 ? row1 : row0) + (tile + (s >> 1) * kGroup + b * 2048u));
  }
  // Elements 32 m .. of each row, rows 16 s .. of the tile: the sum runs over the rows.
  __device__ __forceinline__ typename T::frag column(uint32_t tile, int m, int s) const {
    const uint32_t by = tile + m * kGroup + s * 1024u;
    union {
      s16x4 half[2];
      typename T::frag all;
    } u;
    u.half[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((SDC_LDS s16x4*)(uintptr_t)(col0 + by));
    u.half[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((SDC_LDS s16x4*)(uintptr_t)(col1 + by));
    return u.all;
  }
};

// A row of a matrix as the right operand of a product along it: elements 16 s + 8 half ..
template <class T, int DB>
__device__ __forceinline__ void load_row(const unsigned char* p, bool has, uint32_t d, typename T::frag (&f)[2 * DB]) {
  const uint32_t half = threadIdx.x >> 5 & 1u;
#pragma unroll
  for (int s = 0; s < 2 * DB; ++s) {
    const uint32_t e = 16u * s + 8u * half;
    u32x4 v = {0u, 0u, 0u, 0u};
    if (has && e < d) v = *reinterpret_cast<const u32x4*>(p + 2u * e);
    f[s] = __builtin_bit_cast(typename T::frag, v);
  }
}

// Sets *found where the tile holds an infinity or NaN; each wave looks at its part.
template <class T, int DB, int WAVES>
__device__ __forceinline__ void find_nonfinite(const unsigned char* tile, uint32_t* found) {
  constexpr uint32_t one = std::is_same<T, Bf16>::value ? 0x00800080u : 0x04000400u;  // of the exponent's last bit
  uint32_t bad = 0;
#pragma unroll
  for (uint32_t i = 0; i < tile_bytes<DB>() / (1024u * WAVES); ++i) {
    const u32x4 v = *reinterpret_cast<const u32x4*>(tile + (i * 64u * WAVES + threadIdx.x) * 16u);
    bad |= ((v.x & 0x7FFF7FFFu) + one) | ((v.y & 0x7FFF7FFFu) + one) | ((v.z & 0x7FFF7FFFu) + one) |
           ((v.w & 0x7FFF7FFFu) + one);
  }
  if (__any((bad & 0x80008000u) != 0u)) *found = 1u;
}

// sum_e x_e y_e of two rows.
template <class T>
__device__ __forceinline__ float dot_rows(const unsigned char* x, const unsigned char* y, uint32_t d) {
  float s = 0.0f;
  for (uint32_t e = 0; e < d; e += 8) {
    const u32x4 u = *reinterpret_cast<const u32x4*>(x + 2u * e), v = *reinterpret_cast<const u32x4*>(y + 2u * e);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      s += T::value(u[i] & 0xFFFFu) * T::value(v[i] & 0xFFFFu) + T::value(u[i] >> 16) * T::value(v[i] >> 16);
  }
  return s;
}

// x[i] += w times elements lane and lane + 64 of a row.
template <class T>
__device__ __forceinline__ void add_row(float (&x)[2], float w, const unsigned char* row, uint32_t d) {
  const uint32_t lane = threadIdx.x & 63u;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (lane + 64u * i < d) x[i] += w * T::value(reinterpret_cast<const uint16_t*>(row)[lane + 64u * i]);
}

// Four 16-bit values of consecutive elements.
template <class T>
__device__ __forceinline__ void store4(uint16_t* p, float a, float b, float c, float d) {
  *reinterpret_cast<uint2*>(p) = uint2{T::bits(a) | T::bits(b) << 16, T::bits(c) | T::bits(d) << 16};
}

// fp16: the power of two, less kPShift's, that dS = p (dP - delta) is held times: |dP| and
// |delta| are at most the product of the largest norms of a row of dout and of v, so 2^14
// over twice that keeps dS below fp16's largest number and as far as can be from its
// subnormals.  bf16 has fp32's exponents.
template <class T>
__device__ __forceinline__ int grad_shift(const AttnArgs& a) {
  if constexpr (std::is_same<T, Bf16>::value) return 0;
  float x = 0.0f, y = 0.0f;
  for (uint32_t i = threadIdx.x & 63u; i < kNormParts; i += 64) {
    x = __builtin_fmaxf(x, a.norms[i]);
    y = __builtin_fmaxf(y, a.norms[kNormParts + i]);
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    x = __builtin_fmaxf(x, __shfl_xor(x, off));
    y = __builtin_fmaxf(y, __shfl_xor(y, off));
  }
  const float bits = 0.5f * (__builtin_amdgcn_logf(x) + __builtin_amdgcn_logf(y)) + 1.0f;  // log2 of the bound
  const float e = __builtin_floorf(14.0f - bits);
  return __builtin_amdgcn_readfirstlane((int)__builtin_fminf(__builtin_fmaxf(e, -60.0f), 60.0f));
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// Own loads have landed, own LDS accesses are done, and everyone's.
__device__ __forceinline__ void tile_barrier() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// The part of the scores' fingerprint row that a lane has of a tile: sums of the raw scores'
// 16-bit halves, and weighted by their rows within the tile (and tokens, for dk and dv), in 32
// bits: at most 32 elements of weight below 64.  One dot product of halves does what a 64-bit
// addition or multiplication takes two to four issues for (8192 tokens, 64/8 heads of 128,
// causal: the forward pass with its row takes 1.41 ms, without 1.04; with 64-bit sums it took 2.72).
struct ScoreSums {
  uint32_t lo = 0, hi = 0, wlo = 0, whi = 0, x = 0;
  float odd = 0.0f;  // 0, or NaN where a score was infinite or NaN
};

// Adds a 32 x 32 block, rows 32 n .. of the tile counted from the lane's first; scores that
// do not attend are 0.
__device__ __forceinline__ void add_scores(ScoreSums& c, const f32x16& z, int n) {
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const uint32_t x = __float_as_uint(z[r]), w = 32u * n + element_row(r, 0);
    c.lo = udot2(x, 1u, c.lo);
    c.hi = udot2(x, 1u << 16, c.hi);
    if (w != 0) {
      c.wlo = udot2(x, w, c.wlo);
      c.whi = udot2(x, w << 16, c.whi);
    }
    c.x ^= x;
    c.odd = __builtin_fmaf(z[r], 0.0f, c.odd);
  }
}

__device__ __forceinline__ uint32_t nonfinite_scores(const f32x16& z) {
  uint32_t n = 0;
#pragma unroll
  for (int r = 0; r < 16; ++r) n += __builtin_fabsf(z[r]) < __builtin_inff() ? 0u : 1u;
  return n;
}

// Joins a tile's sums; first: index, from 1, of the lane's first score of the tile, step: of
// the next row.
__device__ __forceinline__ void join_scores(Lane& ln, const ScoreSums& c, uint64_t first, uint64_t step) {
  const uint64_t s = c.lo + ((uint64_t)c.hi << 16);
  ln.s += s;
  ln.w += first * s + step * (c.wlo + ((uint64_t)c.whi << 16));
  ln.x ^= c.x;
}

}  // namespace
}  // namespace sdc
