// gemm_device.h -- the matrix-product tile of the cross-entropy head for
// gfx950: C[m][n] = sum_k A[m][k] B[n][k] for 16-bit A and B whose rows are
// contiguous in k, accumulated in fp32 by MFMA.
//
// A workgroup of 8 waves computes 256 x 256 of C; wave (wm, wn), wm = 0..1,
// wn = 0..3, holds rows 128 wm .. and columns 64 wn .. of it as 8 x 4 tiles of
// 16 x 16 (128 accumulator registers).  k advances 64 at a time through two
// LDS buffers of 64 KiB: the next buffer is filled by direct global-to-LDS
// loads (16 bytes a lane, no registers) while the current one is multiplied.
// Within a 128-byte row of a buffer the eight 16-byte chunks are permuted by
// the row's low three bits, so that the 16 rows x 16 bytes an MFMA operand
// reads at once fall on different banks; direct loads write LDS in lane order,
// so the permutation is made in the addresses they read.
#pragma once

#include "scan_device.h"

namespace sdc {
namespace {

constexpr uint32_t kTile = 256;     // rows and columns of C per workgroup
constexpr uint32_t kTileK = 64;     // k per LDS buffer
constexpr uint32_t kGemmBlock = 512;
constexpr uint32_t kBufBytes = 2 * kTile * kTileK * 2;  // A and B of one k step
constexpr uint32_t kGemmLds = 2 * kBufBytes;

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

// An operand: `rows` rows of K elements, `stride` bytes apart, 16-byte aligned.
struct Operand {
  const unsigned char* p;
  uint64_t stride;
  uint32_t rows;
};

// Where a thread's accumulators stand in the tile: element r of acc[i][j] is
// C[row(i) + r][col(j)].
struct Place {
  uint32_t lane, wm, wn;
  __device__ __forceinline__ Place()
      : lane(threadIdx.x & 63u), wm(threadIdx.x >> 8), wn((threadIdx.x >> 6) & 3u) {}
  __device__ __forceinline__ uint32_t row(int i) const { return wm * 128u + i * 16u + (lane >> 4) * 4u; }
  __device__ __forceinline__ uint32_t col(int j) const { return wn * 64u + j * 16u + (lane & 15u); }
};

#define SDC_LDS __attribute__((address_space(3)))

// Sum over k in [k0, k1) (k0 and the operands' chunks of 8 aligned; k from K on
// reads as zero) of the tile at row m0 of A and row n0 of B.  Rows past the
// operands' last are read as that row: their results mean nothing.
template <class T>
__device__ __forceinline__ void gemm_tile(const Operand& A, const Operand& B, uint32_t m0, uint32_t n0,
                                          uint32_t k0, uint32_t k1, uint32_t K, unsigned char* lds,
                                          f32x4 (&acc)[8][4]) {
  typedef typename T::frag frag;
  const Place at;
  const uint32_t t = threadIdx.x;
  // loads: thread t fills chunk t & 7 of rows t / 8 + 64 i of each operand
  const uint32_t q = (t & 7u) ^ ((t >> 3) & 7u);
  const unsigned char *pa[4], *pb[4];
#pragma unroll
  for (uint32_t i = 0; i < 4; ++i) {
    pa[i] = A.p + (uint64_t)min(m0 + i * 64u + (t >> 3), A.rows - 1u) * A.stride + q * 16u;
    pb[i] = B.p + (uint64_t)min(n0 + i * 64u + (t >> 3), B.rows - 1u) * B.stride + q * 16u;
  }
  const unsigned char* zero = reinterpret_cast<const unsigned char*>(&g_zero16);
  const auto fill = [&](uint32_t k, uint32_t buf) {
    SDC_LDS unsigned char* base =
        (SDC_LDS unsigned char*)(lds + buf * kBufBytes + (t & ~63u) * 16u);
    const bool in = k + q * 8u < K;
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) {
      __builtin_amdgcn_global_load_lds(
          (const SDC_GLOBAL uint32_t*)(in ? pa[i] + (uint64_t)k * 2u : zero),
          (SDC_LDS uint32_t*)(base + i * 8192u), 16, 0, 0);
      __builtin_amdgcn_global_load_lds(
          (const SDC_GLOBAL uint32_t*)(in ? pb[i] + (uint64_t)k * 2u : zero),
          (SDC_LDS uint32_t*)(base + 32768u + i * 8192u), 16, 0, 0);
    }
  };
  // operand reads: row lane & 15 of a 16-row group, chunk 4 s + lane / 16 of its 8
  const uint32_t off = (at.lane & 15u) * 128u + (((at.lane >> 4) ^ (at.lane & 7u)) << 4);
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  fill(k0, 0);
  uint32_t buf = 0;
  for (uint32_t k = k0; k < k1; k += kTileK, buf ^= 1u) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();  // this buffer is whole, and everyone has left the other
    asm volatile("" ::: "memory");
    if (k + kTileK < k1) fill(k + kTileK, buf ^ 1u);
    const unsigned char* sa = lds + buf * kBufBytes + at.wm * 16384u;
    const unsigned char* sb = lds + buf * kBufBytes + 32768u + at.wn * 8192u;
#pragma unroll
    for (uint32_t s = 0; s < 2; ++s) {
      const uint32_t o = off ^ (s * 64u);
      frag a[8], b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const frag*>(sb + j * 2048 + o);
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] = *reinterpret_cast<const frag*>(sa + i * 2048 + o);
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = T::mfma(a[i], b[j], acc[i][j]);
    }
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
