// gemm_device.h -- the matrix-product tile of the cross-entropy head for
// gfx950: C[m][n] = sum_k A(m, k) B(n, k) for 16-bit operands whose rows are
// contiguous either in k or, "k-major", in m (n), accumulated in fp32 by MFMA.
//
// A workgroup computes an M x N tile of C (a Shape): 256 x 256 by 8 waves, 128 x
// 128 or 64 x 64 by 4 where the larger tiles would be too few to fill the chip,
// and 128 x 32 or 64 x 32 by 4 for few rows of B.  Wave (wm, wn) holds M / WM
// rows and N / WN columns of it as I x J groups of 16 x 16 (for 256 x 256: 128
// accumulator registers).
// k advances 64 at a time through two LDS buffers (64 KiB each for 256 x 256):
// the next buffer is filled by direct global-to-LDS loads (16 bytes a lane, no
// registers) while the current one is multiplied.  Four buffers of 32 k instead
// measured 4 to 10 % slower where rows run along k (64-byte pieces of rows) and
// equal where they do not.
// Direct loads write LDS in lane order, so the permutations below, which keep
// the lanes of one LDS read on different banks, are made in the addresses they
// read from.
//   rows along k: rows of 128 bytes; the eight 16-byte chunks of a row are
//     permuted by its low three bits.  An operand register group is one
//     16-byte read per lane.
//   k-major: 64 rows of 2 M (2 N) bytes; their granules of 32 bytes (16 columns)
//     in row k are permuted by f(k) = k & 3 | (k >> 3 & 3) << 2, which differs
//     over the 16 rows that one transposing read takes.  A group is two
//     transposing 8-byte reads (each gives a lane four k of its column), which
//     is what spares transposed copies of the weights, the inputs and dz.
// Measured, 256 x 256, back to back: 2048 x 128256 x 8192 (rows along k, with the
// softmax' statistics) 3.3 to 3.4 ms (1.26 to 1.31 PFLOP/s), the whole gradient of
// that size, two thirds of it k-major products, 10.9 to 11.1 ms (1.17 to 1.19); MFMA
// units 60 % busy at 4096 x 50304 x 2048.  Bound by LDS reads beside the products: a step of 256 x 256 x 64
// reads 192 KiB and multiplies for 2048 cycles.  Four waves of 128 x 128 instead,
// which read a third less, measured 10 to 14 % slower: with one wave a SIMD nothing
// covers its waits.
#pragma once

#include "scan_device.h"

namespace sdc {
namespace {

constexpr uint32_t kTileK = 64;  // k per LDS buffer

template <uint32_t M_, uint32_t N_, uint32_t WM_, uint32_t WN_, uint32_t DEEP = 0, bool LATE = false>
struct Shape {
  static constexpr uint32_t M = M_, N = N_, WM = WM_, WN = WN_;
  static constexpr uint32_t kDeep = DEEP;  // steps in flight of gemm_tile_deep
  static constexpr bool kLate = LATE;      // the next step's loads stand behind LDS reads (see gemm_step)
  static constexpr uint32_t kThreads = 64 * WM * WN;
  static constexpr int I = M / WM / 16, J = N / WN / 16;
  static constexpr uint32_t kA = M * kTileK * 2, kBuf = (M + N) * kTileK * 2;  // bytes of A, of both, of one k step
  static constexpr uint32_t kLds = 2 * kBuf;
};
typedef Shape<256, 256, 2, 4, 0, true> BigTile;
typedef Shape<128, 128, 2, 2> SmallTile;
typedef Shape<64, 64, 2, 2> TinyTile;
typedef Shape<128, 32, 4, 1, 3> FewTile;
typedef Shape<64, 32, 4, 1, 4> FewTinyTile;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

struct Bf16 {
  typedef bf16x8 frag;
  // dz is at most 1 in magnitude and bf16 has fp32's exponents
  static constexpr float kDzScale = 1.0f;
  static __device__ __forceinline__ f32x4 mfma(frag a, frag b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ uint32_t bits(float x) {
    return __builtin_bit_cast(unsigned short, (__bf16)x);
  }
};

struct Fp16 {
  typedef f16x8 frag;
  // probabilities of 1e-5 would be subnormal in fp16: dz is held 2^15 times as large
  static constexpr float kDzScale = 32768.0f;
  static __device__ __forceinline__ f32x4 mfma(frag a, frag b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ uint32_t bits(float x) {
    return __builtin_bit_cast(unsigned short, (_Float16)x);
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
template <class S>
struct Place {
  uint32_t lane, wm, wn;
  __device__ __forceinline__ Place()
      : lane(threadIdx.x & 63u), wm((threadIdx.x >> 6) / S::WN), wn((threadIdx.x >> 6) % S::WN) {}
  __device__ __forceinline__ uint32_t row(int i) const { return wm * (S::M / S::WM) + i * 16u + (lane >> 4) * 4u; }
  __device__ __forceinline__ uint32_t col(int j) const { return wn * (S::N / S::WN) + j * 16u + (lane & 15u); }
};

#define SDC_LDS __attribute__((address_space(3)))
typedef short s16x4 __attribute__((ext_vector_type(4)));

// 16 bytes per lane from src to LDS at base + 16 * lane (base uniform).  Written
// as an instruction of its own: the compiler otherwise waits for all loads in
// flight before every transposing read of LDS, whichever buffer it reads.  It
// writes no register but m0, the address; gemm_tile waits for it with vmcnt(0).
// The compiler reserves m0, so it warns that a clobber of m0 is not undone: nor
// need it be, as whatever reads m0 sets it first.  (Restoring m0 in the statement
// instead measured 0.3 to 1.3 % slower.)
__device__ __forceinline__ void load_to_lds(const unsigned char* src, uint32_t base) {
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %1, off"
      :
      : "s"(base), "v"(src)
      : "m0", "memory");
#pragma clang diagnostic pop
}

// How A's rows may lie: at 16-byte boundaries (kAt16), read straight into LDS;
// or anywhere (kAny: rows of at least 8 elements at any even address, of any
// length), read through registers, which direct loads to LDS cannot.  kDeep:
// anywhere, and both operands through registers, several steps ahead (see
// gemm_tile_deep).
enum RowsAt : int { kAt16, kAny, kDeep };

// Sixteen bytes at any even address.
__device__ __forceinline__ u32x4 load16_any(const unsigned char* p) {
  typedef uint32_t vec __attribute__((ext_vector_type(4), aligned(2)));
  return *(const SDC_GLOBAL vec*)p;
}

// v moved down by n 16-bit elements (0..7), zeros above: the last chunk of a
// row of a length not divisible by 8, read as the row's last 16 bytes.  In 32-bit
// steps, as a 64-bit shift by a register must not stand here: with the amount in
// the last register of the wave's allocation (v239 of 240, say) this chip reads
// another amount now and then, and the compiler does place it there.
__device__ __forceinline__ u32x4 drop_elements(u32x4 v, uint32_t n) {
  if (n & 4u) v = u32x4{v.z, v.w, 0u, 0u};
  if (n & 2u) v = u32x4{v.y, v.z, v.w, 0u};
  const uint32_t bits = (n & 1u) * 16u;
  return u32x4{__builtin_amdgcn_alignbit(v.y, v.x, bits), __builtin_amdgcn_alignbit(v.z, v.y, bits),
               __builtin_amdgcn_alignbit(v.w, v.z, bits), v.w >> bits};
}

// One operand's side of the tile: its loads into LDS, step after step, and its
// reads.
template <class T, uint32_t ROWS, uint32_t THREADS, bool KMAJOR, RowsAt AT>
struct Side {
  static constexpr uint32_t kLoads = ROWS * 8 / THREADS;  // 16-byte loads of a thread per step
  static constexpr uint32_t kRow = 2 * ROWS;              // bytes of a k-major row
  static constexpr uint32_t kPass = THREADS * 16;         // bytes that one load of every thread fills
  static constexpr uint32_t kGranules = ROWS / 16 - 1;
  static constexpr uint32_t kPassK = THREADS * 8 / ROWS;  // k-major: rows of k that they fill
  static_assert(kLoads * THREADS == ROWS * 8, "the loads cover a step");
  const unsigned char* p[kLoads];  // of the thread's loads of the next step
  uint64_t step;                   // bytes from one step to the next
  uint32_t limit;                  // k from here on reads as zero
  uint32_t k_in;                   // k of the thread's first load within a step
  uint32_t off;                    // of the lane's LDS reads
  uint32_t drop[kLoads];           // kAny, k-major: elements past the end of the rows that a load starts before

  // at0: first row of C's index; base: LDS row (rows along k) or granule
  // (k-major) of the wave's first group.  Rows along k past the operand's last
  // are read as the last, chunks past a k-major one's columns as its last eight.
  __device__ __forceinline__ void init(const Operand& o, uint32_t at0, uint32_t base, uint32_t k0) {
    const uint32_t t = threadIdx.x, lane = t & 63u;
    if constexpr (KMAJOR) {
      limit = o.rows;
      k_in = t / (ROWS / 8);
      step = o.stride * kTileK;
#pragma unroll
      for (uint32_t i = 0; i < kLoads; ++i) {
        const uint32_t k = i * kPassK + k_in, f = (k & 3u) | ((k >> 3) & 3u) << 2;
        const uint32_t col = at0 + ((((t % (ROWS / 8)) >> 1) ^ (f & kGranules)) * 16u) + (t & 1u) * 8u;
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
      for (uint32_t i = 0; i < kLoads; ++i)
        p[i] = o.p + (uint64_t)min(at0 + i * (THREADS / 8) + (t >> 3), o.rows - 1u) * o.stride + (uint64_t)(k0 + k_in) * 2u;
      off = (base + (lane & 15u)) * 128u + (((lane >> 4) ^ (lane & 7u)) << 4);
    }
  }
  // Starts the loads of the operand's part of step k, into LDS at byte `dst`
  // (kAt16) or into held, which settle writes to LDS; called step by step.
  __device__ __forceinline__ void fill(uint32_t k, uint32_t dst, u32x4 (&held)[kLoads]) {
    if constexpr (AT == kAt16) {
      const uint32_t base = dst + __builtin_amdgcn_readfirstlane(threadIdx.x & ~63u) * 16u;
      if (k + kTileK <= limit) {
#pragma unroll
        for (uint32_t i = 0; i < kLoads; ++i) load_to_lds(p[i], base + i * kPass);
      } else {
        const unsigned char* zero = reinterpret_cast<const unsigned char*>(&g_zero16);
#pragma unroll
        for (uint32_t i = 0; i < kLoads; ++i)
          load_to_lds(k + k_in + (KMAJOR ? i * kPassK : 0u) < limit ? p[i] : zero, base + i * kPass);
      }
    } else if (AT == kAny && k + kTileK <= limit) {
#pragma unroll
      for (uint32_t i = 0; i < kLoads; ++i) held[i] = load16_any(p[i]);
    } else {
      // Chunks past the end come from the zero vector; one that ends past its
      // row starts at the row's last 16 bytes.  kDeep takes this path at every
      // step and shifts them in settle: with no branch around the loads and no
      // use of them here, the waits count exactly the younger ones.
      const unsigned char* zero = reinterpret_cast<const unsigned char*>(&g_zero16);
      const uint32_t back = past_end(k);
#pragma unroll
      for (uint32_t i = 0; i < kLoads; ++i) {
        const bool in = k + k_in + (KMAJOR ? i * kPassK : 0u) < limit;
        held[i] = load16_any(in ? p[i] - back * 2u : zero);
        if (AT == kAny && !KMAJOR) held[i] = drop_elements(held[i], back);
      }
    }
#pragma unroll
    for (uint32_t i = 0; i < kLoads; ++i) p[i] += step;
  }
  // Rows along k: elements past the row's end in the thread's chunk of step k
  // (below 8 for a chunk that has any of the row's).
  __device__ __forceinline__ uint32_t past_end(uint32_t k) const {
    const uint32_t at = k + k_in;
    return !KMAJOR && at < limit && at + 8u > limit ? at + 8u - limit : 0u;
  }
  __device__ __forceinline__ void settle(uint32_t k, const u32x4 (&held)[kLoads], unsigned char* dst) const {
    if constexpr (AT != kAt16) {
#pragma unroll
      for (uint32_t i = 0; i < kLoads; ++i) {
        u32x4 v = held[i];
        if constexpr (KMAJOR || AT == kDeep) {
          const uint32_t n = KMAJOR ? drop[i] : past_end(k);
          if (__any(n != 0u)) v = drop_elements(v, n);
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

// The products of a step from LDS at la and lb; during(s) is called between the
// reads of half s of the step and their products.  Where one workgroup fills a CU
// (kLate, 256 x 256) the next step's loads are issued there, so that the LDS reads
// start right behind the barrier (2048 x 8192 x 128256: 3330 us; with the loads
// first 3760; with both halves read first 3450), and the products of k-major
// operands go before other waves' work (PRIO; with / without: the gradient of that
// size 10.9 ms / 11.2; rows along k, the loss, 3390 us / 3330).  In the smaller
// tiles another workgroup covers the reads, and both cost (loss, loads first / late:
// 755 x 5296 x 688 49 us / 55, with the row 100 x 2048 x 50304 45 / 49 and 800 x
// 2048 x 50304 199 / 226; gradient 4096 x 256 x 12800 128 / 142, 600 x 1024 x 20000
// 102 / 113; 64 x 2048 x 50304 alone 41.6 / 40.7).
template <class T, class S, bool PRIO, class SA, class SB, class F>
__device__ __forceinline__ void gemm_step(const SA& sa, const SB& sb, const unsigned char* la,
                                          const unsigned char* lb, f32x4 (&acc)[S::I][S::J], F&& during) {
#pragma unroll
  for (uint32_t s = 0; s < 2; ++s) {
    typename T::frag a[S::I], b[S::J];
#pragma unroll
    for (int j = 0; j < S::J; ++j) b[j] = sb.read(lb, j, s);
#pragma unroll
    for (int i = 0; i < S::I; ++i) a[i] = sa.read(la, i, s);
    during(s);
    if constexpr (PRIO) __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int i = 0; i < S::I; ++i)
#pragma unroll
      for (int j = 0; j < S::J; ++j) acc[i][j] = T::mfma(a[i], b[j], acc[i][j]);
    if constexpr (PRIO) __builtin_amdgcn_s_setprio(0);
  }
}

// gemm_tile for few rows of B, where a step lasts as long as the loads it waits
// for: three steps (four in the 64-row tile) of both operands are in flight, in
// registers, of which there are plenty.  Same operations in the same order, so the same bits.  k1 is where
// the operands end.
template <class T, class S>
__device__ __forceinline__ void gemm_tile_deep(const Operand& A, const Operand& B, uint32_t m0, uint32_t n0,
                                               uint32_t k0, uint32_t k1, unsigned char* lds,
                                               f32x4 (&acc)[S::I][S::J]) {
  const Place<S> at;
  Side<T, S::M, S::kThreads, false, kDeep> sa;
  Side<T, S::N, S::kThreads, false, kDeep> sb;
  sa.init(A, m0, at.wm * (S::M / S::WM), k0);
  sb.init(B, n0, at.wn * (S::N / S::WN), k0);
#pragma unroll
  for (int i = 0; i < S::I; ++i)
#pragma unroll
    for (int j = 0; j < S::J; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  u32x4 ha[S::kDeep][sa.kLoads], hb[S::kDeep][sb.kLoads];  // step k of every kDeep in set k % kDeep
#pragma unroll
  for (uint32_t i = 0; i < S::kDeep; ++i) {
    sa.fill(k0 + i * kTileK, 0, ha[i]);
    sb.fill(k0 + i * kTileK, 0, hb[i]);
  }
  sa.settle(k0, ha[0], lds);
  sb.settle(k0, hb[0], lds + S::kA);
  uint32_t buf = 0;
  // Steps past the last, up to a multiple of kDeep, multiply zeros: no sum that
  // starts at +0 changes by them.
  for (uint32_t k = k0; k < k1; k += S::kDeep * kTileK) {
#pragma unroll
    for (uint32_t i = 0; i < S::kDeep; ++i) {
      const uint32_t next = (i + 1) % S::kDeep, at_k = k + i * kTileK;
      // own writes of this buffer and reads of the other are done (a barrier that
      // also waited for the loads in flight would undo them)
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      __builtin_amdgcn_s_barrier();  // this buffer is whole, and everyone has left the other
      asm volatile("" ::: "memory");
      sa.fill(at_k + S::kDeep * kTileK, 0, ha[i]);
      sb.fill(at_k + S::kDeep * kTileK, 0, hb[i]);
      __builtin_amdgcn_sched_barrier(0);  // the loads go first
      gemm_step<T, S, false>(sa, sb, lds + buf * S::kBuf, lds + buf * S::kBuf + S::kA, acc, [](uint32_t) {});
      buf ^= 1u;
      sa.settle(at_k + kTileK, ha[next], lds + buf * S::kBuf);
      sb.settle(at_k + kTileK, hb[next], lds + buf * S::kBuf + S::kA);
    }
  }
  __syncthreads();  // the buffers may be reused
}

// Sum over k in [k0, k1) (k0 a multiple of 64) of the tile at row m0 of A's
// index and n0 of B's.  What the tile holds past either's last means nothing.
// AAT: how A's rows lie; B's lie at 16-byte boundaries.
template <class T, class S, RowsAt AAT, bool AK, bool BK>
__device__ __forceinline__ void gemm_tile(const Operand& A, const Operand& B, uint32_t m0, uint32_t n0,
                                          uint32_t k0, uint32_t k1, unsigned char* lds,
                                          f32x4 (&acc)[S::I][S::J]) {
  if constexpr (AAT == kDeep) {
    static_assert(!AK && !BK, "rows along k");
    gemm_tile_deep<T, S>(A, B, m0, n0, k0, k1, lds, acc);
  } else {
    const Place<S> at;
    Side<T, S::M, S::kThreads, AK, AAT> sa;
    Side<T, S::N, S::kThreads, BK, kAt16> sb;
    sa.init(A, m0, at.wm * (S::M / S::WM) / (AK ? 16u : 1u), k0);
    sb.init(B, n0, at.wn * (S::N / S::WN) / (BK ? 16u : 1u), k0);
    const uint32_t lds0 = (uint32_t)(uintptr_t)(SDC_LDS unsigned char*)lds;
#pragma unroll
    for (int i = 0; i < S::I; ++i)
#pragma unroll
      for (int j = 0; j < S::J; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    u32x4 ha[sa.kLoads], hb[sb.kLoads];  // ha: kAny, A's loads of the next step; hb is not used
    const auto fill = [&](uint32_t k, uint32_t buf) {
      sa.fill(k, lds0 + buf * S::kBuf, ha);
      sb.fill(k, lds0 + buf * S::kBuf + S::kA, hb);
    };
    fill(k0, 0);
    sa.settle(k0, ha, lds);
    uint32_t buf = 0;
    for (uint32_t k = k0; k < k1; k += kTileK, buf ^= 1u) {
      // own loads have landed, own reads and writes of the other buffer are done
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
      __builtin_amdgcn_s_barrier();  // this buffer is whole, and everyone has left the other
      asm volatile("" ::: "memory");
      const unsigned char* la = lds + buf * S::kBuf;
      if (!S::kLate && k + kTileK < k1) fill(k + kTileK, buf ^ 1u);
      gemm_step<T, S, S::kLate && AK>(sa, sb, la, la + S::kA, acc, [&](uint32_t s) {
        if (!S::kLate || k + kTileK >= k1) return;
        if (s == 0) sa.fill(k + kTileK, lds0 + (buf ^ 1u) * S::kBuf, ha);
        else sb.fill(k + kTileK, lds0 + (buf ^ 1u) * S::kBuf + S::kA, hb);
      });
      if (k + kTileK < k1) sa.settle(k + kTileK, ha, lds + (buf ^ 1u) * S::kBuf);
    }
    __syncthreads();  // the buffers may be reused
  }
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
