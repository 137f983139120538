// adamw_device.h -- device and plan definitions of the AdamW step over a
// tensor list (the optimizer step that the weight check of AWS Machine
// Learning Blog, "Detecting and recovering from silent data corruption on
// Amazon SageMaker HyperPod", section "Check 3", runs after).
#pragma once

#include "fingerprint_device.h"

namespace sdc {

constexpr uint64_t kAdamwMagic = 0x31766D6164414453ull;  // "SDAdamv1", little-endian

// A tensor is cut into items of one round of loads of a workgroup each (a
// multiple of the 128-element block of an 8-bit state).  One round, because what
// hides the memory's latency here is the number of waves that load: longer
// items measured 4921 / 5130 / 5200 us at 4096 / 16384 / 65536 elements, this size
// 4826 us (0.96B fp32 weights).  Tensors of up to a wave's round are items of one
// wave: with waves for up to 2048 / 1024 / 512 / 128 elements, lists of small
// tensors measured 607 / 601 / 596 / 589 us (20,000 of up to 65536 elements) and 92 /
// 86 / 83 / 82 us (4,000, 8-bit states); below a round a wave's lanes idle.
constexpr uint64_t kAdamwItemElems = 2048;
constexpr uint64_t kAdamwWaveElems = 512;

// Elements that share one scale byte of an 8-bit state.
constexpr uint32_t kStateBlock = 128;

// Kernel classes by the widths of what they stream: param 0 fp32, 1 16-bit,
// 2 16-bit with fp32 master weights; grad 0 fp32, 1 16-bit; state 0 fp32,
// 1 8-bit.
constexpr uint32_t kAdamwClasses = 12;
constexpr uint32_t adamw_class(uint32_t param, uint32_t grad, uint32_t state) {
  return (param * 2 + grad) * 2 + state;
}

struct AdamwDesc {
  void* param;
  const void* grad;  // null: the tensor is left as it is
  void* exp_avg;
  void* exp_avg_sq;
  float* master;
  uint8_t* exp_avg_scale;
  uint8_t* exp_avg_sq_scale;
  uint64_t first;  // elements of the list before this tensor (the random bits' counter)
  uint32_t group;
  uint32_t param_dtype, grad_dtype;
  uint32_t pad;
};
static_assert(sizeof(AdamwDesc) == 80, "AdamW descriptor layout");

struct AdamwItem {
  uint64_t start;   // first element
  uint32_t len;     // elements
  uint32_t tensor;  // descriptor, and row, of the tensor
  uint32_t slot;    // partial-row slot (tensors of several items)
  uint32_t whole;   // 1: the item is the whole tensor and stores its row
  uint64_t pad;
};
static_assert(sizeof(AdamwItem) == 32, "AdamW item layout");

// What the gate of a step leaves for its items: the factor of the gradients,
// whether the step is skipped, and the keys of its random bits.
struct AdamwGate {
  float scale;
  uint32_t skip;
  uint32_t k0, k1;
};

struct AdamwCoef {
  float beta1, omb1, beta2, omb2;  // omb = 1 - beta
  float size;                      // lr / (1 - beta1^t)
  float rbc2;                      // 1 / sqrt(1 - beta2^t)
  float eps, decay;                // decay = 1 - lr * weight_decay
};
static_assert(sizeof(AdamwCoef) == 32, "AdamW coefficients");

// Device plan: [AdamwGate][coefficients x n_groups][descriptors x n_tensors]
// [items][split entries] (pad to 256) [partial rows].
struct AdamwOffsets {
  uint64_t gate, coef, desc, items, split, partials, end;
};

inline AdamwOffsets adamw_offsets(uint64_t n_tensors, uint64_t n_groups, uint64_t n_items,
                                  uint64_t n_split, uint64_t n_slots) {
  AdamwOffsets o;
  o.gate = 0;
  o.coef = 64;
  o.desc = o.coef + n_groups * sizeof(AdamwCoef);
  o.items = o.desc + n_tensors * sizeof(AdamwDesc);
  o.items = (o.items + 31) / 32 * 32;
  o.split = o.items + n_items * sizeof(AdamwItem);
  o.partials = (o.split + n_split * sizeof(PlanSplit) + 255) / 256 * 256;
  o.end = o.partials + n_slots * sizeof(sdc_row);
  return o;
}

struct AdamwArgs {
  const AdamwGate* gate;
  const AdamwCoef* coef;
  const AdamwDesc* desc;
  const AdamwItem* items;  // of the class: n_block workgroup items, then n_wave wave items
  uint32_t n_block, n_wave;
  sdc_row* partials;
  sdc_row* rows;  // null: no rows
};

// Launches the class's items (csrc/adamw32.hip, csrc/adamw8.hip).
int32_t launch_adamw32(uint32_t cls, const AdamwArgs& a, hipStream_t s);
int32_t launch_adamw8(uint32_t cls, const AdamwArgs& a, hipStream_t s);

namespace {

// Loads through the constant address space: what the plan holds does not
// change while a step's kernels run, so uniform reads of it are scalar loads
// that stores in between do not repeat.
template <class T>
__device__ __forceinline__ T load_const(const T* p) {
  struct Words {
    uint32_t w[sizeof(T) / 4];
  } x;
#pragma unroll
  for (uint32_t i = 0; i < sizeof(T) / 4; ++i) x.w[i] = ((const __attribute__((address_space(4))) uint32_t*)p)[i];
  return __builtin_bit_cast(T, x);
}

// An item's streams, each from the item's first element on.
struct AdamwStreams {
  unsigned char *param, *exp_avg, *exp_avg_sq, *master, *exp_avg_scale, *exp_avg_sq_scale;
  const unsigned char* grad;
};

// Vectors at any element alignment: the hardware's global accesses need no
// more (they split only where a vector crosses a cache line).
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));
typedef uint32_t u32_any __attribute__((aligned(1)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// W dwords at p, streamed (every byte of the step is touched once).
template <int W>
__device__ __forceinline__ void load_words(const void* p, uint32_t (&w)[W]) {
  const unsigned char* c = (const unsigned char*)p;
  if constexpr (W >= 4) {
#pragma unroll
    for (int i = 0; i < W; i += 4) {
      const u32x4_any v = __builtin_nontemporal_load((const SDC_GLOBAL u32x4_any*)(c + 4 * i));
      w[i] = v.x;
      w[i + 1] = v.y;
      w[i + 2] = v.z;
      w[i + 3] = v.w;
    }
  } else if constexpr (W == 2) {
    const u32x2_any v = __builtin_nontemporal_load((const SDC_GLOBAL u32x2_any*)c);
    w[0] = v.x;
    w[1] = v.y;
  } else {
    w[0] = __builtin_nontemporal_load((const SDC_GLOBAL u32_any*)c);
  }
}

template <int W>
__device__ __forceinline__ void store_words(void* p, const uint32_t (&w)[W]) {
  unsigned char* c = (unsigned char*)p;
  if constexpr (W >= 4) {
#pragma unroll
    for (int i = 0; i < W; i += 4) {
      const u32x4_any v = {w[i], w[i + 1], w[i + 2], w[i + 3]};
      __builtin_nontemporal_store(v, (SDC_GLOBAL u32x4_any*)(c + 4 * i));
    }
  } else if constexpr (W == 2) {
    const u32x2_any v = {w[0], w[1]};
    __builtin_nontemporal_store(v, (SDC_GLOBAL u32x2_any*)c);
  } else {
    __builtin_nontemporal_store(w[0], (SDC_GLOBAL u32_any*)c);
  }
}

// One vector of E elements of ES bytes as packed little-endian words, of
// which those from `lo` on and below `hi` are the item's (0 and E: all of
// them; hi <= lo: none).  The others read as zero and are not written.
template <int E, int ES>
struct Vec {
  static constexpr int W = E * ES / 4;
  uint32_t w[W];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ void load(const unsigned char* base, uint32_t at, int lo, int hi) {
    const unsigned char* p = base + at * ES;
    if (lo <= 0 && hi >= E) {
      load_words<W>(p, w);
      return;
    }
    zero();
    if (lo >= hi) return;
    // element loads from addresses held inside the range, all in flight together
    uint32_t x[E];
#pragma unroll
    for (int k = 0; k < E; ++k) x[k] = (uint32_t)load_elem<ES>(p + min(max(k, lo), hi - 1) * ES);
#pragma unroll
    for (int k = 0; k < E; ++k)
      if (k >= lo && k < hi) w[k * ES / 4] |= x[k] << (8 * ((k * ES) & 3));
  }
  // zeroes the elements below lo and from hi on
  __device__ __forceinline__ void cut(int lo, int hi) {
#pragma unroll
    for (int k = 0; k < E; ++k)
      if (k < lo || k >= hi)
        w[k * ES / 4] &= ES == 4 ? 0u : ~(((1u << (8 * ES & 31)) - 1u) << (8 * ((k * ES) & 3)));
  }
  __device__ __forceinline__ void store(unsigned char* base, uint32_t at, int lo, int hi) const {
    unsigned char* p = base + at * ES;
    if (lo <= 0 && hi >= E) {
      store_words<W>(p, w);
      return;
    }
#pragma unroll
    for (int k = 0; k < E; ++k)
      if (k >= lo && k < hi) {
        const uint32_t x = w[k * ES / 4] >> (8 * ((k * ES) & 3));
        if constexpr (ES == 4) *(SDC_GLOBAL uint32_t*)(p + k * 4) = x;
        else if constexpr (ES == 2) *(SDC_GLOBAL uint16_t*)(p + k * 2) = (uint16_t)x;
        else *(SDC_GLOBAL uint8_t*)(p + k) = (uint8_t)x;
      }
  }
};

__device__ __forceinline__ float bf16_to_float(uint32_t h) { return __uint_as_float(h << 16); }
__device__ __forceinline__ float f16_to_float(uint32_t h) {
  return (float)__builtin_bit_cast(_Float16, (unsigned short)h);
}

// Round to nearest, ties to even: the rounding of torch's own casts, off by at
// most half a step.  NaN stays NaN (quieted).
__device__ __forceinline__ uint32_t float_to_bf16(float x) {
  const __bf16 b = (__bf16)x;
  return __builtin_bit_cast(unsigned short, b);
}
__device__ __forceinline__ uint32_t float_to_f16(float x) {
  const _Float16 h = (_Float16)x;
  return __builtin_bit_cast(unsigned short, h);
}

template <int E, int ES>
__device__ __forceinline__ void to_floats(const Vec<E, ES>& v, bool half, float (&f)[E]) {
  if constexpr (ES == 4) {
#pragma unroll
    for (int k = 0; k < E; ++k) f[k] = __uint_as_float(v.w[k]);
  } else if (half) {
#pragma unroll
    for (int k = 0; k < E; ++k) f[k] = f16_to_float((v.w[k / 2] >> (16 * (k & 1))) & 0xFFFFu);
  } else {
#pragma unroll
    for (int k = 0; k < E; ++k)
      f[k] = (k & 1) ? __uint_as_float(v.w[k / 2] & 0xFFFF0000u) : bf16_to_float(v.w[k / 2]);
  }
}

template <int E, int ES>
__device__ __forceinline__ void from_floats(const float (&f)[E], bool half, Vec<E, ES>& v) {
  if constexpr (ES == 4) {
#pragma unroll
    for (int k = 0; k < E; ++k) v.w[k] = __float_as_uint(f[k]);
  } else if (half) {
#pragma unroll
    for (int k = 0; k < E; k += 2) v.w[k / 2] = float_to_f16(f[k]) | (float_to_f16(f[k + 1]) << 16);
  } else {
#pragma unroll
    for (int k = 0; k < E; k += 2) v.w[k / 2] = float_to_bf16(f[k]) | (float_to_bf16(f[k + 1]) << 16);
  }
}

// Fingerprint of the new weights while they are in registers: the lane's
// sums over its vectors of E elements, vector i of the item being lane
// i % LANES's, as in the scan: a = sum x, c = sum k x (k: slot in the vector),
// q = the running sum of a after each vector.
template <int E, int ES>
struct RowAcc {
  typedef std::conditional_t<(ES == 2), uint32_t, uint64_t> sum_t;
  sum_t a = 0, c = 0;
  uint64_t q = 0;
  uint32_t x = 0, nf = 0;
  __device__ __forceinline__ void add(const Vec<E, ES>& v, uint32_t m2, uint32_t k2) {
#pragma unroll
    for (int i = 0; i < Vec<E, ES>::W; ++i) {
      const uint32_t d = v.w[i];
      if constexpr (ES == 2) {
        a = udot2(d, 0x00010001u, a);
        c = udot2(d, (uint32_t)((2 * i + 1) << 16 | (2 * i)), c);
        nf += (uint32_t)__builtin_popcount(((d & m2) + k2) & 0x80008000u);
      } else {
        a += d;
        c += (uint64_t)i * d;
        nf += ((d & 0x7F800000u) + 0x00800000u) >> 31;
      }
      x ^= d;
    }
    q += a;
  }
  // T: vectors of the lane, those past the end counted as zero vectors; shift:
  // places before the item's first element in its first vector
  __device__ __forceinline__ Lane lane(uint32_t l, uint32_t lanes, uint64_t T, uint32_t shift) const {
    Lane ln;
    ln.s = a;
    ln.w = ((uint64_t)(1u + E * l) - shift) * a + (uint64_t)(lanes * E) * (T * a - q) + c;
    ln.x = x;
    ln.nf = nf;
    return ln;
  }
};

__device__ __forceinline__ void store_row(sdc_row* dst, const Lane& ln, uint64_t w) {
  ulonglong2* d = reinterpret_cast<ulonglong2*>(dst);
  d[0] = ulonglong2{ln.s, w};
  d[1] = ulonglong2{ln.x, ln.nf};
}

// The fp32 number nearest to sqrt(v), for v = 0, v >= 2^-96, Inf or NaN (below,
// within one unit in the last place): the hardware's root s is off by at most
// one unit, and the signs of v - s s' for s' its neighbours below and above
// tell which of the three it is (each an fma, exact in sign as long as it
// does not underflow).
__device__ __forceinline__ float sqrt_nearest(float v) {
  const float s = __builtin_amdgcn_sqrtf(v);
  const float below = __uint_as_float(__float_as_uint(s) - 1u), above = __uint_as_float(__float_as_uint(s) + 1u);
  float r = s;
  if (__builtin_fmaf(-below, s, v) <= 0.0f) r = below;
  if (__builtin_fmaf(-above, s, v) > 0.0f) r = above;
  return r;
}

// One step of one element, in fp32: m, v and the weight p of the gradient g
// (scaled already); returns sqrt(v).  The quotient takes the hardware's
// reciprocal, and EXACT false also its square root (each off by about one unit
// in the last place, which moves the update, not the weight, by 2^-23 of
// itself).  EXACT: every operation of m, v and sqrt(v) is rounded on its own,
// so the 8-bit codes drawn from them follow from the formulas, whoever
// computes them.
template <bool EXACT>
__device__ __forceinline__ float adamw_element(const AdamwCoef& c, float g, float& m, float& v, float& p) {
  float r;
  if constexpr (EXACT) {
    {
#pragma clang fp contract(off)
      m = m * c.beta1 + g * c.omb1;
      v = v * c.beta2 + (g * g) * c.omb2;
    }
    r = sqrt_nearest(v);
  } else {
    m = __builtin_fmaf(c.beta1, m, c.omb1 * g);
    v = __builtin_fmaf(c.beta2, v, c.omb2 * (g * g));
    r = __builtin_amdgcn_sqrtf(v);
  }
  const float q = m * __builtin_amdgcn_rcpf(__builtin_fmaf(r, c.rbc2, c.eps));
  p = __builtin_fmaf(-c.size, q, p * c.decay);
  return r;
}

// The two streams of state of E elements of an item.
template <int E>
struct State32 {
  Vec<E, 4> m, v;
  __device__ __forceinline__ void load(const AdamwStreams& d, uint32_t at, int lo, int hi) {
    m.load(d.exp_avg, at, lo, hi);
    v.load(d.exp_avg_sq, at, lo, hi);
  }
  template <class F, class G>
  __device__ __forceinline__ void update(F&& element, G&& done, uint64_t, const AdamwGate&, bool) {
#pragma unroll
    for (int k = 0; k < E; ++k) {
      float mk = __uint_as_float(m.w[k]), vk = __uint_as_float(v.w[k]);
      element(k, mk, vk);
      m.w[k] = __float_as_uint(mk);
      v.w[k] = __float_as_uint(vk);
    }
    done();
  }
  __device__ __forceinline__ void store(const AdamwStreams& d, uint32_t at, int lo, int hi) const {
    m.store(d.exp_avg, at, lo, hi);
    v.store(d.exp_avg_sq, at, lo, hi);
  }
};

// Largest value over groups of G (16 or 32) adjacent lanes, in all of them.
template <int G>
__device__ __forceinline__ uint32_t group_umax(uint32_t x) {
  x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0xB1, 0xF, 0xF, true));   // lane ^ 1
  x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x4E, 0xF, 0xF, true));   // lane ^ 2
  x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x141, 0xF, 0xF, true));  // mirrored in 8
  x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x140, 0xF, 0xF, true));  // mirrored in 16
  if constexpr (G == 32) x = max(x, (uint32_t)__shfl_xor((int)x, 16));
  return x;
}

// States in 8 bits.  A block of 128 elements of the tensor shares the power
// of two 2^(s-127), s = max(exponent field of the block's largest magnitude
// - 7, 1): the largest lands in [128, 256), so rounding up never reaches
// e4m3's NaN.  m is held as e4m3 codes of m / 2^(s-127), v as those of
// sqrt(v) / 2^(s-127) (a square root halves the range of exponents that 8
// bits have to span).  e4m3 has the bits of an fp32 number 2^-120 times as
// large, cut to 3 mantissa bits, subnormals included.
//
// Codes are 1/8 to 1/16 apart, a step moves a state by 1 - beta (0.1 .. 0.001)
// of itself: rounding to nearest would never move v.  So each code is drawn
// from its two neighbours with the element's random bits, for m so that the
// expected value is m, for sqrt(v) so that the expected square is v; the
// moving averages then stay unbiased.  A v above zero is never held as zero
// (the quotient would be m / eps).  NaN and Inf become NaN.
template <int E>
struct State8 {
  static constexpr int kLanes = kStateBlock / E;  // lanes of a block
  Vec<E, 1> m, v;
  uint32_t ms, vs;  // scale bytes
  __device__ __forceinline__ void load(const AdamwStreams& d, uint32_t at, int lo, int hi) {
    m.load(d.exp_avg, at, lo, hi);
    v.load(d.exp_avg_sq, at, lo, hi);
    ms = vs = 0;
    if (hi > 0) {
      ms = ((const SDC_GLOBAL uint8_t*)d.exp_avg_scale)[at / kStateBlock];
      vs = ((const SDC_GLOBAL uint8_t*)d.exp_avg_sq_scale)[at / kStateBlock];
    }
  }
  static __device__ __forceinline__ uint32_t hash(uint32_t lo, uint32_t hi_key, uint32_t k0) {
    // Two multiply-xorshift rounds; multipliers and shifts of least bias from
    // the search published by C. Wellons ("Prospecting for Hash Functions").
    uint32_t a = lo + k0;
    a = (a ^ (a >> 16)) * 0x7FEB352Du;
    a ^= hi_key;
    a = (a ^ (a >> 15)) * 0x846CA68Bu;
    return a ^ (a >> 16);
  }
  template <class F, class G>
  __device__ __forceinline__ void update(F&& element, G&& done, uint64_t index, const AdamwGate& gate, bool wraps) {
    const float md = __uint_as_float(ms << 23), vd = __uint_as_float(vs << 23);  // scale byte 0: zeros
    float mf[E], rf[E], mtop = 0.0f, rtop = 0.0f;  // NaNs are left out of the largest
#pragma unroll
    for (int k = 0; k < E; k += 2) {
      const f32x2 a = (k & 2) ? __builtin_amdgcn_cvt_pk_f32_fp8((int)m.w[k / 4], true)
                              : __builtin_amdgcn_cvt_pk_f32_fp8((int)m.w[k / 4], false);
      const f32x2 b = (k & 2) ? __builtin_amdgcn_cvt_pk_f32_fp8((int)v.w[k / 4], true)
                              : __builtin_amdgcn_cvt_pk_f32_fp8((int)v.w[k / 4], false);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float rk = b[j] * vd;
        float vk = rk * rk;
        mf[k + j] = a[j] * md;
        rf[k + j] = element(k + j, mf[k + j], vk);
        mtop = __builtin_fmaxf(mtop, __builtin_fabsf(mf[k + j]));
        rtop = __builtin_fmaxf(rtop, rf[k + j]);
      }
    }
    ms = scale_byte(group_umax<kLanes>(__float_as_uint(mtop)));
    vs = scale_byte(group_umax<kLanes>(__float_as_uint(rtop)));
    done();  // the weights are final: stored before the codes are drawn
    const uint32_t hk = gate.k1 + (uint32_t)(index >> 32) * 0x2C1B3C6Du;
    // `wraps` is uniform: whether the low word of the element counter wraps inside the item
    if (wraps) codes<true>(mf, rf, (uint32_t)index, hk, gate.k0);
    else codes<false>(mf, rf, (uint32_t)index, hk, gate.k0);
  }
  // The codes of the E new m and sqrt(v) with the scale bytes ms and vs.
  template <bool WRAPS>
  __device__ __forceinline__ void codes(const float (&mf)[E], const float (&rf)[E], uint32_t lo0, uint32_t hk,
                                        uint32_t k0) {
    const float mu = __uint_as_float((254u - ms) << 23), ru = __uint_as_float((254u - vs) << 23);  // 1 / 2^(s-127)
#pragma unroll
    for (int w = 0; w < E / 4; ++w) {
      uint32_t h[4], cm = 0, cv = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = 4 * w + i;
        const uint32_t lo = lo0 + k;
        h[i] = hash(lo, (WRAPS && lo < lo0) ? hk + 0x2C1B3C6Du : hk, k0);
        const float t = rf[k] * ru;
        uint32_t c = __float_as_uint(__builtin_amdgcn_ldexpf(t, -120)) >> 20;
        const f32x2 r = __builtin_amdgcn_cvt_pk_f32_fp8((int)(c * 257u + 256u), false);  // codes c, c + 1
        const float u = __builtin_fmaf((float)(h[i] >> 16), 0x1p-16f, 0x1p-17f);
        {
#pragma clang fp contract(off)
          // 4-bit numbers: their squares, the difference and u times it are exact
          const float lo_v = r.x * r.x;
          const float gap = u * __builtin_fmaf(r.y, r.y, -lo_v);
          c += gap < t * t - lo_v ? 1u : 0u;
        }
        c = umed3(c, min(__float_as_uint(rf[k]), 1u), 0x7Fu);  // c in 1 .. 0x7F, or 0 for a zero
        cv |= c << (8 * i);
      }
      // m: the hardware's stochastic rounding adds the seed below the kept
      // bits and cuts; here 16 random bits and a half of the next
      cm = (uint32_t)__builtin_amdgcn_cvt_sr_fp8_f32(mf[4 * w] * mu, (h[0] << 16) | 0x8000u, (int)cm, 0);
      cm = (uint32_t)__builtin_amdgcn_cvt_sr_fp8_f32(mf[4 * w + 1] * mu, (h[1] << 16) | 0x8000u, (int)cm, 1);
      cm = (uint32_t)__builtin_amdgcn_cvt_sr_fp8_f32(mf[4 * w + 2] * mu, (h[2] << 16) | 0x8000u, (int)cm, 2);
      cm = (uint32_t)__builtin_amdgcn_cvt_sr_fp8_f32(mf[4 * w + 3] * mu, (h[3] << 16) | 0x8000u, (int)cm, 3);
      m.w[w] = cm;
      v.w[w] = cv;
    }
  }
  static __device__ __forceinline__ uint32_t umed3(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("v_med3_u32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
  }
  static __device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
    return (uint32_t)max((int)(top >> 23) - 7, 1);
  }
  __device__ __forceinline__ void store(const AdamwStreams& d, uint32_t at, int lo, int hi) const {
    m.store(d.exp_avg, at, lo, hi);
    v.store(d.exp_avg_sq, at, lo, hi);
    if (hi > 0 && at % kStateBlock == 0) {
      ((SDC_GLOBAL uint8_t*)d.exp_avg_scale)[at / kStateBlock] = (uint8_t)ms;
      ((SDC_GLOBAL uint8_t*)d.exp_avg_sq_scale)[at / kStateBlock] = (uint8_t)vs;
    }
  }
};

template <uint32_t PARAM, uint32_t GRAD, uint32_t STATE, bool ROWS>
struct AdamwCfg {
  static constexpr int kParamBytes = PARAM == 0 ? 4 : 2;
  static constexpr int kGradBytes = GRAD == 0 ? 4 : 2;
  static constexpr bool kMaster = PARAM == 2;
  static constexpr bool kRows = ROWS;
  static constexpr bool kState8 = STATE == 1;
  static constexpr bool kExact = STATE == 1;
  // Elements per lane and vector: 16 bytes of the widest stream.
  static constexpr int E = (STATE == 0 || PARAM != 1 || GRAD == 0) ? 4 : 8;
  static constexpr int U = 8 / E;  // vectors per lane and round
  typedef std::conditional_t<STATE == 0, State32<E>, State8<E>> State;
};

// One item by LANES lanes (256: a workgroup, 64: a wave).
template <class Cfg, uint32_t LANES>
__device__ __forceinline__ void adamw_item(const AdamwArgs& a, const AdamwItem& it, uint32_t l) {
  constexpr int E = Cfg::E, U = Cfg::U;
  const AdamwDesc desc = load_const(a.desc + it.tensor);
  const AdamwGate gate = load_const(a.gate);
  const AdamwCoef coef = load_const(a.coef + desc.group);
  // fp32 states: vectors are counted from the 16-byte boundary at or below the
  // item's first element of exp_avg (a tensor's later items start on one), so
  // that lists packed at odd offsets stream aligned: the other fp32 streams
  // usually share the offset.
  const uint32_t shift =
      Cfg::kState8 ? 0u : ((uint32_t)((uintptr_t)desc.exp_avg >> 2) + (uint32_t)it.start) & 3u;
  const uint64_t from = it.start - shift;
  AdamwStreams d;
  d.param = (unsigned char*)desc.param + from * Cfg::kParamBytes;
  d.grad = (const unsigned char*)desc.grad + from * Cfg::kGradBytes;
  d.exp_avg = (unsigned char*)desc.exp_avg + from * (Cfg::kState8 ? 1 : 4);
  d.exp_avg_sq = (unsigned char*)desc.exp_avg_sq + from * (Cfg::kState8 ? 1 : 4);
  d.master = (unsigned char*)desc.master + from * 4;
  d.exp_avg_scale = desc.exp_avg_scale + from / kStateBlock;
  d.exp_avg_sq_scale = desc.exp_avg_sq_scale + from / kStateBlock;
  const uint64_t first = desc.first + it.start;
  const bool phalf = desc.param_dtype == SDC_F16, ghalf = desc.grad_dtype == SDC_F16;
  const bool skip = gate.skip != 0 || desc.grad == nullptr;
  const bool wraps = (uint32_t)first + it.len < it.len;
  const uint32_t m2 = phalf ? 0x7C007C00u : 0x7F807F80u, k2 = phalf ? 0x04000400u : 0x00800080u;
  if (skip && !Cfg::kRows) return;
  RowAcc<E, Cfg::kParamBytes> acc;
  // A round: U vectors per lane from vector v0.  FULL: every lane's vectors
  // are whole, so all loads are issued with no branch between them.
  struct Round {
    Vec<E, Cfg::kParamBytes> p[U];
    Vec<E, Cfg::kGradBytes> g[U];
    Vec<E, 4> mw[U];
    typename Cfg::State st[U];
  };
  constexpr uint32_t kRound = LANES * U;
  const uint32_t end = it.len + shift, rounds = (end + kRound * E - 1) / (kRound * E);
  const auto lo = [&](uint32_t j, auto full) { return decltype(full)::value ? 0 : (int)shift - (int)j; };
  const auto hi = [&](uint32_t j, auto full) { return decltype(full)::value ? E : (int)end - (int)j; };
  const auto load = [&](Round& r, uint32_t v0, auto full) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t j = (v0 + u * LANES + l) * E;
      r.g[u].load(d.grad, j, lo(j, full), hi(j, full));
      if constexpr (Cfg::kMaster) r.mw[u].load(d.master, j, lo(j, full), hi(j, full));
      else r.p[u].load(d.param, j, lo(j, full), hi(j, full));
      r.st[u].load(d, j, lo(j, full), hi(j, full));
    }
  };
  const auto step = [&](Round& r, uint32_t v0, auto full) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t j = (v0 + u * LANES + l) * E;
      float gf[E], pf[E];
      to_floats(r.g[u], ghalf, gf);
      if constexpr (Cfg::kMaster) to_floats(r.mw[u], false, pf);
      else to_floats(r.p[u], phalf, pf);
      r.st[u].update(
          [&](int k, float& m, float& v) {
            return adamw_element<Cfg::kExact>(coef, gf[k] * gate.scale, m, v, pf[k]);
          },
          [&]() {
            if constexpr (Cfg::kMaster) {
              from_floats(pf, false, r.mw[u]);
              r.mw[u].store(d.master, j, lo(j, full), hi(j, full));
            }
            from_floats(pf, phalf, r.p[u]);
            if (Cfg::kRows && !decltype(full)::value) r.p[u].cut(lo(j, full), hi(j, full));
            r.p[u].store(d.param, j, lo(j, full), hi(j, full));
            if constexpr (Cfg::kRows) acc.add(r.p[u], m2, k2);
          },
          first - shift + j, gate, wraps);
      r.st[u].store(d, j, lo(j, full), hi(j, full));
    }
  };
  const std::true_type whole;
  const std::false_type part;
  const uint32_t T = rounds * U;
  if (skip) {  // the weights stay: their row alone
    for (uint32_t i = 0; i < T; ++i) {
      const uint32_t j = (i * LANES + l) * E;
      Vec<E, Cfg::kParamBytes> p;
      p.load(d.param, j, lo(j, part), hi(j, part));
      acc.add(p, m2, k2);
    }
  } else {
    for (uint32_t i = 0; i < rounds; ++i) {
      Round r;
      if ((i > 0 || shift == 0) && (i + 1) * kRound * E <= end) {
        load(r, i * kRound, whole);
        step(r, i * kRound, whole);
      } else {
        load(r, i * kRound, part);
        step(r, i * kRound, part);
      }
    }
  }
  if constexpr (Cfg::kRows) {
    Lane ln = acc.lane(l, LANES, T, shift);
    if constexpr (LANES == 64) wave_reduce(ln);
    else block_reduce(ln);
    if (l != 0) return;
    ln.x = finish_xor<TypeTag<Cfg::kParamBytes, false, kChkNone>>(ln.x);
    store_row(it.whole ? a.rows + it.tensor : a.partials + it.slot, ln, ln.w + it.start * ln.s);
  }
}

// The items of a class: workgroup items first, then four wave items a workgroup.
// Bound by memory: 0.96B fp32 weights with fp32 states (28 bytes each) 4.9 ms (5.5
// TB/s), bf16 with 8-bit states (10 bytes) 1.8 ms back to back (5.4 TB/s, next to as
// much vector arithmetic; 2.0 ms on average in a trace).  With rows 4.8 and 2.2 ms.
template <class Cfg>
__global__ void __launch_bounds__(kBlock) adamw_kernel(const AdamwArgs a) {
  if (blockIdx.x < a.n_block) {
    adamw_item<Cfg, kBlock>(a, load_const(a.items + blockIdx.x), threadIdx.x);
    return;
  }
  const uint32_t w =
      __builtin_amdgcn_readfirstlane((blockIdx.x - a.n_block) * kWaves + (threadIdx.x >> 6));
  if (w < a.n_wave) adamw_item<Cfg, 64>(a, load_const(a.items + (a.n_block + w)), threadIdx.x & 63u);
}

template <uint32_t PARAM, uint32_t GRAD, uint32_t STATE>
int32_t launch_adamw_class(const AdamwArgs& a, hipStream_t s) {
  const dim3 grid(a.n_block + (a.n_wave + kWaves - 1) / kWaves), block(kBlock);
  if (a.rows)
    hipLaunchKernelGGL((adamw_kernel<AdamwCfg<PARAM, GRAD, STATE, true>>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((adamw_kernel<AdamwCfg<PARAM, GRAD, STATE, false>>), grid, block, 0, s, a);
  return launch_status();
}

template <uint32_t STATE>
int32_t launch_adamw_state(uint32_t cls, const AdamwArgs& a, hipStream_t s) {
  switch (cls / 2) {
    case 0: return launch_adamw_class<0, 0, STATE>(a, s);
    case 1: return launch_adamw_class<0, 1, STATE>(a, s);
    case 2: return launch_adamw_class<1, 0, STATE>(a, s);
    case 3: return launch_adamw_class<1, 1, STATE>(a, s);
    case 4: return launch_adamw_class<2, 0, STATE>(a, s);
    default: return launch_adamw_class<2, 1, STATE>(a, s);
  }
}

}  // namespace
}  // namespace sdc
