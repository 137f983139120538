// gemm_device.h -- the matrix-product tile of the cross-entropy head for
// gfx950: C[m][n] = sum_k A(m, k) B(n, k) for 16-bit operands whose rows are
// contiguous either in k or, "k-major", in m (n), accumulated in fp32 by MFMA.
//
// A workgroup computes a TILE x TILE tile of C, TILE 256 (8 waves) or, where
// those would be too few to fill the chip, 128 (4 waves).  Wave (wm, wn),
// wm = 0..1, wn = 0..TILE / 64 - 1, holds rows wm TILE / 2 .. and columns
// 64 wn .. of it as TILE / 32 x 4 groups of 16 x 16 (for 256: 128 accumulator
// registers).  k advances 64 at a time through two LDS buffers (64 KiB each
// for 256): the next buffer is filled by direct global-to-LDS loads (16 bytes
// a lane, no registers) while the current one is multiplied.  Four buffers of
// 32 k instead measured 4 to 10 % slower where rows run along k (64-byte
// pieces of rows) and equal where they do not.
// Direct loads write LDS in lane order, so the permutations below, which keep
// the lanes of one LDS read on different banks, are made in the addresses they
// read from.
//   rows along k: TILE rows of 128 bytes; the eight 16-byte chunks of a row are
//     permuted by its low three bits.  An operand register group is one
//     16-byte read per lane.
//   k-major: 64 rows of 2 TILE bytes; the TILE / 16 granules of 32 bytes
//     (16 columns) of row k are permuted by f(k) = k & 3 | (k >> 3 & 3) << 2,
//     which differs over the 16 rows that one transposing read takes.  A group
//     is two transposing 8-byte reads (each gives a lane four k of its column),
//     which is what spares transposed copies of the weights, the inputs and dz.
// Measured alone on random data, TILE 256: 4096 x 32768 x 2048 (rows along k)
// 431 us (1275 TFLOP/s), 2048 x 32768 x 4096 (k-major) 455 us (1210).
#pragma once

#include "scan_device.h"

namespace sdc {
namespace {

constexpr uint32_t kTileK = 64;  // k per LDS buffer
constexpr uint32_t gemm_block(uint32_t tile) { return 2 * tile; }              // threads
constexpr uint32_t buf_bytes(uint32_t tile) { return 2 * tile * kTileK * 2; }  // A and B of one k step
constexpr uint32_t gemm_lds(uint32_t tile) { return 2 * buf_bytes(tile); }

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

struct Bf16 {
  typedef bf16x8 frag;
  static constexpr uint32_t kDtype = SDC_BF16;
  // dz is at most 1 in magnitude and bf16 has fp32's exponents
  static constexpr float kDzScale = 1.0f;
  static __device__ __forceinline__ f32x4 mfma(frag a, frag b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ uint32_t bits(float x) {
    return __builtin_bit_cast(unsigned short, (__bf16)x);
  }
  static __device__ __forceinline__ float value(uint32_t b) { return __uint_as_float(b << 16); }
};

struct Fp16 {
  typedef f16x8 frag;
  static constexpr uint32_t kDtype = SDC_F16;
  // probabilities of 1e-5 would be subnormal in fp16: dz is held 2^15 times as large
  static constexpr float kDzScale = 32768.0f;
  static __device__ __forceinline__ f32x4 mfma(frag a, frag b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ uint32_t bits(float x) {
    return __builtin_bit_cast(unsigned short, (_Float16)x);
  }
  static __device__ __forceinline__ float value(uint32_t b) {
    return (float)__builtin_bit_cast(_Float16, (unsigned short)b);
  }
};

// An operand with `rows` rows (of C's index, or, k-major, of k), `stride` bytes
// apart, each of `cols` elements: 16-byte aligned with cols a multiple of 8, or
// (RowsAt kAny) at any even address with cols at least 8.
struct Operand {
  const unsigned char* p;
  uint64_t stride;
  uint32_t rows, cols;
};

// Where a thread's accumulators stand in the tile: element r of acc[i][j] is
// C[row(i) + r][col(j)].
template <uint32_t TILE>
struct Place {
  uint32_t lane, wm, wn;
  __device__ __forceinline__ Place()
      : lane(threadIdx.x & 63u), wm(threadIdx.x / TILE), wn((threadIdx.x >> 6) & (TILE / 64u - 1u)) {}
  __device__ __forceinline__ uint32_t row(int i) const { return wm * (TILE / 2) + i * 16u + (lane >> 4) * 4u; }
  __device__ __forceinline__ uint32_t col(int j) const { return wn * 64u + j * 16u + (lane & 15u); }
};

#define SDC_LDS __attribute__((address_space(3)))
typedef short s16x4 __attribute__((ext_vector_type(4)));

// 16 bytes per lane from src to LDS at base + 16 * lane (base uniform).  Written
// as an instruction of its own: the compiler otherwise waits for all loads in
// flight before every transposing read of LDS, whichever buffer it reads.  It
// has no output register; gemm_tile waits for it with vmcnt(0).  m0 is a
// register the compiler reserves and writes right before each use of its own.
__device__ __forceinline__ void load_to_lds(const unsigned char* src, uint32_t base) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %1, off"
      :
      : "s"(base), "v"(src)
      : "memory");
}

// How an operand's rows may lie: at 16-byte boundaries (kAt16), read straight
// into LDS; or anywhere (kAny: rows of at least 8 elements at any even address,
// of any length), read through registers, which direct loads to LDS cannot.
enum RowsAt : int { kAt16, kAny };

// Sixteen bytes at any even address.
__device__ __forceinline__ u32x4 load16_any(const unsigned char* p) {
  typedef uint32_t vec __attribute__((ext_vector_type(4), aligned(2)));
  return *(const SDC_GLOBAL vec*)p;
}

// v moved down by n 16-bit elements (0..7), zeros above: the last chunk of a
// row of a length not divisible by 8, read as the row's last 16 bytes.
__device__ __forceinline__ u32x4 drop_elements(u32x4 v, uint32_t n) {
  const uint64_t lo = lohi(v.x, v.y), hi = lohi(v.z, v.w);
  const uint32_t bits = (n & 3u) * 16u;
  const uint64_t a = n < 4u ? lo : hi, b = n < 4u ? hi : 0ull;
  const uint64_t rl = bits ? (a >> bits) | (b << (64u - bits)) : a, rh = b >> bits;
  return u32x4{(uint32_t)rl, (uint32_t)(rl >> 32), (uint32_t)rh, (uint32_t)(rh >> 32)};
}

// One operand's side of the tile: its loads into LDS, step after step, and its
// reads.
template <class T, uint32_t TILE, bool KMAJOR, RowsAt AT>
struct Side {
  static constexpr uint32_t kRow = 2 * TILE;         // bytes of a k-major row
  static constexpr uint32_t kPass = 2 * TILE * 16;   // bytes that one load of every thread fills
  static constexpr uint32_t kGranules = TILE / 16 - 1;
  const unsigned char* p[4];  // of the thread's loads of the next step
  uint64_t step;              // bytes from one step to the next
  uint32_t limit;             // k from here on reads as zero
  uint32_t k_in;              // k of the thread's first load within a step
  uint32_t off;               // of the lane's LDS reads
  uint32_t drop[4];           // kAny, k-major: elements past the end of the rows that a load starts before
  u32x4 held[4];              // kAny: the loads of the next step

  // at0: first row of C's index; base: LDS row (rows along k) or granule
  // (k-major) of the wave's first group.  Rows along k past the operand's last
  // are read as the last, chunks past a k-major one's columns as its last eight.
  __device__ __forceinline__ void init(const Operand& o, uint32_t at0, uint32_t base, uint32_t k0) {
    const uint32_t t = threadIdx.x, lane = t & 63u;
    if constexpr (KMAJOR) {
      limit = o.rows;
      k_in = t / (TILE / 8);
      step = o.stride * kTileK;
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i) {
        const uint32_t k = i * 16u + k_in, f = (k & 3u) | ((k >> 3) & 3u) << 2;
        const uint32_t col = at0 + ((((t % (TILE / 8)) >> 1) ^ (f & kGranules)) * 16u) + (t & 1u) * 8u;
        const uint32_t from = min(col, o.cols - 8u);
        p[i] = o.p + (uint64_t)(k0 + k) * o.stride + (uint64_t)from * 2u;
        drop[i] = min(col - from, 7u);
      }
      const uint32_t g = lane >> 4, r = (lane >> 2) & 3u, f = r | g << 2;
      off = (8u * g + r) * kRow + ((base ^ (f & kGranules)) << 5) + (lane & 3u) * 8u;
    } else {
      limit = o.cols;
      const uint32_t q = (t & 7u) ^ ((t >> 3) & 7u);
      k_in = q * 8u;
      step = kTileK * 2u;
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i)
        p[i] = o.p + (uint64_t)min(at0 + i * (TILE / 4) + (t >> 3), o.rows - 1u) * o.stride + (uint64_t)(k0 + k_in) * 2u;
      off = (base + (lane & 15u)) * 128u + (((lane >> 4) ^ (lane & 7u)) << 4);
    }
  }
  // Starts the loads of the operand's part of step k into LDS at byte `dst`;
  // called step by step.
  __device__ __forceinline__ void fill(uint32_t k, uint32_t dst) {
    if constexpr (AT == kAt16) {
      const uint32_t base = dst + __builtin_amdgcn_readfirstlane(threadIdx.x & ~63u) * 16u;
      if (k + kTileK <= limit) {
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) load_to_lds(p[i], base + i * kPass);
      } else {
        const unsigned char* zero = reinterpret_cast<const unsigned char*>(&g_zero16);
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i)
          load_to_lds(k + k_in + (KMAJOR ? i * 16u : 0u) < limit ? p[i] : zero, base + i * kPass);
      }
    } else if (k + kTileK <= limit) {
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i) held[i] = load16_any(p[i]);
    } else if constexpr (KMAJOR) {
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i) {
        held[i] = u32x4{0u, 0u, 0u, 0u};
        if (k + k_in + i * 16u < limit) held[i] = load16_any(p[i]);
      }
    } else {
      // chunks that end past the row start at its last 16 bytes; those past it are zero
      const uint32_t at = k + k_in, back = at + 8u > limit ? min(at + 8u - limit, 8u) : 0u;
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i) {
        held[i] = u32x4{0u, 0u, 0u, 0u};
        if (at < limit) held[i] = drop_elements(load16_any(p[i] - back * 2u), back & 7u);
      }
    }
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) p[i] += step;
  }
  // kAny: writes what fill has loaded to LDS at `dst`.
  __device__ __forceinline__ void settle(unsigned char* dst) const {
    if constexpr (AT == kAny) {
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i) {
        u32x4 v = held[i];
        if constexpr (KMAJOR) {
          if (__any(drop[i] != 0u)) v = drop_elements(v, drop[i]);
        }
        *reinterpret_cast<u32x4*>(dst + i * kPass + threadIdx.x * 16u) = v;
      }
    }
  }
  // Group i (16 rows of C's index) of k 32 s .. of the step in LDS at `src`.
  __device__ __forceinline__ typename T::frag read(const unsigned char* src, int i, uint32_t s) const {
    if constexpr (KMAJOR) {
      const unsigned char* q = src + (off ^ ((uint32_t)i << 5)) + s * (32u * kRow);
      union {
        s16x4 half[2];
        typename T::frag all;
      } u;
      u.half[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((SDC_LDS s16x4*)q);
      u.half[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((SDC_LDS s16x4*)(q + 4 * kRow));
      return u.all;
    } else {
      return *reinterpret_cast<const typename T::frag*>(src + (off ^ (s * 64u)) + i * 2048);
    }
  }
};

// Sum over k in [k0, k1) (k0 a multiple of 64) of the tile at row m0 of A's
// index and n0 of B's.  What the tile holds past either's last means nothing.
// AAT: how A's rows lie; B's lie at 16-byte boundaries.
template <class T, uint32_t TILE, RowsAt AAT, bool AK, bool BK>
__device__ __forceinline__ void gemm_tile(const Operand& A, const Operand& B, uint32_t m0, uint32_t n0,
                                          uint32_t k0, uint32_t k1, unsigned char* lds,
                                          f32x4 (&acc)[TILE / 32][4]) {
  constexpr int kI = TILE / 32;
  constexpr uint32_t kBufBytes = buf_bytes(TILE);
  typedef typename T::frag frag;
  const Place<TILE> at;
  Side<T, TILE, AK, AAT> sa;
  Side<T, TILE, BK, kAt16> sb;
  sa.init(A, m0, AK ? at.wm * (TILE / 32) : at.wm * (TILE / 2), k0);
  sb.init(B, n0, BK ? at.wn * 4u : at.wn * 64u, k0);
  const uint32_t lds0 = (uint32_t)(uintptr_t)(SDC_LDS unsigned char*)lds;
#pragma unroll
  for (int i = 0; i < kI; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const auto fill = [&](uint32_t k, uint32_t buf) {
    sa.fill(k, lds0 + buf * kBufBytes);
    sb.fill(k, lds0 + buf * kBufBytes + kBufBytes / 2);
  };
  fill(k0, 0);
  sa.settle(lds);
  uint32_t buf = 0;
  for (uint32_t k = k0; k < k1; k += kTileK, buf ^= 1u) {
    // own loads have landed, own reads and writes of the other buffer are done
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();  // this buffer is whole, and everyone has left the other
    asm volatile("" ::: "memory");
    if (k + kTileK < k1) fill(k + kTileK, buf ^ 1u);
    const unsigned char* la = lds + buf * kBufBytes;
    const unsigned char* lb = la + kBufBytes / 2;
#pragma unroll
    for (uint32_t s = 0; s < 2; ++s) {
      frag a[kI], b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = sb.read(lb, j, s);
#pragma unroll
      for (int i = 0; i < kI; ++i) a[i] = sa.read(la, i, s);
#pragma unroll
      for (int i = 0; i < kI; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = T::mfma(a[i], b[j], acc[i][j]);
    }
    if (k + kTileK < k1) sa.settle(lds + (buf ^ 1u) * kBufBytes);
  }
  __syncthreads();  // the buffers may be reused
}

// Tile of workgroup b of the nm x nn tiles of C: each XCD (workgroups go to
// them round-robin) takes a contiguous run of the tiles, `nn` fastest, so that
// the tiles an XCD's L2 serves at one time share their rows of A.
__device__ __forceinline__ uint32_t xcd_run(uint32_t b, uint32_t n, uint32_t xcds) {
  if (xcds <= 1u) return b;
  const uint32_t per = n / xcds, extra = n % xcds, x = b % xcds, i = b / xcds;
  return x * per + min(x, extra) + i;
}

}  // namespace
}  // namespace sdc
