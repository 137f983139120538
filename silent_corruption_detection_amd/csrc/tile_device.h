// tile_device.h -- what the kernels around the matrix-product tile share: their
// epilogues' staging, the tiles' fingerprint rows, and on the host the rules that choose
// tiles and splits.
#pragma once

#include <algorithm>
#include <type_traits>

#include "fingerprint_device.h"
#include "gemm_device.h"

namespace sdc {

// Copies the R x C matrix src (rows `stride` bytes apart, elements at any even
// address) to dst [R][c_pad], zeros from column C on.  mask: rows whose target
// is outside [0, vocab) become zeros, whatever they hold.
struct PackArgs {
  const unsigned char* src;
  uint64_t stride;
  uint32_t R, C, c_pad;
  uint16_t* dst;
  const int64_t* mask;
  uint64_t vocab;
};
int32_t launch_pack(const PackArgs& a, hipStream_t s);

// A matrix' row from its tiles' rows; with ref, a difference under col_mask adds 1
// to *mismatch.
int32_t launch_merge_tile_rows(const sdc_row* parts, uint32_t n, const sdc_row* ref, uint32_t col_mask, sdc_row* row,
                               uint32_t* mismatch, hipStream_t s);

// n 16-bit zeros (a fill kernel).
int32_t launch_zero16(uint16_t* p, uint64_t n, hipStream_t s);

// CUs that the rules below fill.  The MI355X' number, not the current device's: tiles,
// pieces and splits follow from the sizes alone, so the results' bits and the
// workspace (asked for without a device) are the same on a part of the chip.
constexpr uint32_t kCus = 256;

// Tokens of the tiles for few of them.
constexpr uint32_t kFew = FewTile::N;

// Tiles of one launch: a grid has fewer than 2^32 threads.
constexpr uint32_t kLaunchTiles = 1u << 22;

constexpr uint64_t up(uint64_t x, uint64_t m) { return (x + m - 1) / m * m; }

uint32_t tiles(uint64_t n, uint32_t tile);
uint32_t logit_tile(uint64_t n, uint64_t vocab);
uint32_t few_rows(uint64_t vocab);

namespace {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.693147180559945309417f;
// 16-bit elements of a staged row of M, padded off the banks
template <class S>
constexpr uint32_t stage_row() { return S::M + 8; }
template <class S>
constexpr uint32_t lds_bytes() { return std::max(S::kLds, S::N * stage_row<S>() * 2); }
static_assert(lds_bytes<BigTile>() + 1024 <= 160u * 1024u, "one workgroup fits a CU");

typedef uint32_t u32x4_at2 __attribute__((ext_vector_type(4), aligned(2)));

// Eight 16-bit elements to any even address, or the first n of them.
__device__ __forceinline__ void store8(uint16_t* p, const uint16_t* s, uint32_t n) {
  if (n >= 8u) {
    *reinterpret_cast<u32x4_at2*>(p) = *reinterpret_cast<const u32x4*>(s);
  } else {
    for (uint32_t e = 0; e < n; ++e) p[e] = s[e];
  }
}

// The part of a wave's lanes of a tile's fingerprint row, joined over the workgroup's WAVES waves.
template <int WAVES>
__device__ __forceinline__ void store_tile_row(Lane ln, sdc_row* out) {
  wave_reduce(ln);
  __shared__ uint64_t waves[4][WAVES];
  const uint32_t wave = threadIdx.x >> 6;
  if ((threadIdx.x & 63u) == 0) {
    waves[0][wave] = ln.s;
    waves[1][wave] = ln.w;
    waves[2][wave] = ln.x;
    waves[3][wave] = ln.nf;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 1; i < WAVES; ++i) {
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

// f(type)
template <class F>
int32_t for_dtype(uint32_t dtype, F&& f) {
  return dtype == SDC_BF16 ? f(Bf16()) : f(Fp16());
}

}  // namespace
}  // namespace sdc
