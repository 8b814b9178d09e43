// mp_tile8.cuh — device building blocks of the block operators that read and
// write 8-bit tensors with scales (mp_norm.cu, mp_swiglu.cu).
//
// The unit of work is 16 consecutive elements of a row in one thread: 32 bytes
// of 16-bit input in two 16-byte loads, and exactly one 16-byte store of FP8
// codes.  A 1x128 tile is then eight lanes and a 1x32 block two, so a tile
// maximum takes three shuffles (one for 1x32) and no shared memory.
#pragma once

#include "mp_device.cuh"

namespace mp {

enum { XF32 = 0, XF16 = 1, XBF16 = 2 };  // the values of mp_dtype

constexpr int kUnit = 16;               // elements per unit
constexpr int kTile = 128;              // elements per FP32 scale
constexpr int kTileLanes = kTile / kUnit;

// One unit as loaded: 16 elements of type XT.
template <int XT>
struct Unit {
  static constexpr int kBytes = kUnit * (XT == XF32 ? 4 : 2);
  static constexpr int kVecs = kBytes / 16;
  uint4 v[kVecs];

  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) v[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  // unit `u` of the row that starts at `row`
  __device__ __forceinline__ void load(const void* row, int64_t u) {
    const unsigned char* p = static_cast<const unsigned char*>(row) + u * kBytes;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) v[i] = ld_cs(p + 16 * i);
  }
  __device__ __forceinline__ void store(void* row, int64_t u) const {
    unsigned char* p = static_cast<unsigned char*>(row) + u * kBytes;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) st_cs(p + 16 * i, v[i]);
  }
  __device__ __forceinline__ uint32_t word(int k) const {  // k a constant after unrolling
    const uint4 q = v[k >> 2];
    return (k & 3) == 0 ? q.x : (k & 3) == 1 ? q.y : (k & 3) == 2 ? q.z : q.w;
  }
  __device__ __forceinline__ void set_word(int k, uint32_t w) {
    uint4& q = v[k >> 2];
    ((k & 3) == 0 ? q.x : (k & 3) == 1 ? q.y : (k & 3) == 2 ? q.z : q.w) = w;
  }
  // elements 2k and 2k + 1
  __device__ __forceinline__ float2 pair(int k) const {
    if constexpr (XT == XF32)
      return make_float2(__uint_as_float(word(2 * k)), __uint_as_float(word(2 * k + 1)));
    else if constexpr (XT == XF16)
      return make_float2(f16lo(word(k)), f16hi(word(k)));
    else
      return make_float2(bf16lo(word(k)), bf16hi(word(k)));
  }
  __device__ __forceinline__ void floats(float (&f)[kUnit]) const {
#pragma unroll
    for (int k = 0; k < kUnit / 2; ++k) {
      const float2 p = pair(k);
      f[2 * k] = p.x;
      f[2 * k + 1] = p.y;
    }
  }
  // rounds to XT, to nearest even
  __device__ __forceinline__ void set_pair(int k, float a, float b) {
    if constexpr (XT == XF32) {
      set_word(2 * k, __float_as_uint(a));
      set_word(2 * k + 1, __float_as_uint(b));
    } else {
      set_word(k, XT == XF16 ? pack_f16x2(a, b) : pack_bf16x2(a, b));
    }
  }
  __device__ __forceinline__ void set(const float (&f)[kUnit]) {
#pragma unroll
    for (int k = 0; k < kUnit / 2; ++k) set_pair(k, f[2 * k], f[2 * k + 1]);
  }
  // the sign bit of element i as stored (a conversion may drop a NaN's sign)
  __device__ __forceinline__ uint32_t sign80(int i) const {
    if constexpr (XT == XF32) return (word(i) >> 24) & 0x80u;
    return (word(i >> 1) >> ((i & 1) ? 24 : 8)) & 0x80u;
  }
};

// 16 weights of a vector of any of the three types (uniform branch).  The
// vector is read again for every row: default caching keeps it in L1.
__device__ __forceinline__ void load_weights(const void* w, int wt, int u, float (&f)[kUnit]) {
  if (wt == XF32) {
    const float4* p = static_cast<const float4*>(w) + u * 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 q = __ldg(p + i);
      f[4 * i] = q.x, f[4 * i + 1] = q.y, f[4 * i + 2] = q.z, f[4 * i + 3] = q.w;
    }
  } else {
    const uint4* p = static_cast<const uint4*>(w) + u * 2;
    Unit<XBF16> r;
    r.v[0] = __ldg(p);
    r.v[1] = __ldg(p + 1);
    if (wt == XBF16) {
      r.floats(f);
    } else {
      Unit<XF16> h;
      h.v[0] = r.v[0];
      h.v[1] = r.v[1];
      h.floats(f);
    }
  }
}

// NaN-propagating max |v| of a unit, as ordered bits (NaN above infinity).
__device__ __forceinline__ uint32_t unit_amax(const float (&v)[kUnit]) {
  float a = 0.0f, b = 0.0f;
#pragma unroll
  for (int i = 0; i < kUnit; i += 2) {
    a = max_abs_nan(a, v[i]);
    b = max_abs_nan(b, v[i + 1]);
  }
  return amax_bits(max_abs_nan(a, b));
}

template <bool E5M2>
__device__ __forceinline__ uint4 cast_unit(const float (&v)[kUnit], float mul) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float a = __fmul_rn(v[4 * k], mul), b = __fmul_rn(v[4 * k + 1], mul);
    const float c = __fmul_rn(v[4 * k + 2], mul), d = __fmul_rn(v[4 * k + 3], mul);
    w[k] = E5M2 ? cvt_e5m2x2(a, b) | (cvt_e5m2x2(c, d) << 16) : cvt_e4m3x2(a, b) | (cvt_e4m3x2(c, d) << 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Codes of a unit in a tile that holds an infinity or a NaN: 0x7F with the
// element's sign for each of those, a zero with its sign for a finite element.
template <typename SignOf>
__device__ __forceinline__ uint4 nonfinite_unit(const float (&v)[kUnit], SignOf sign80) {
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < kUnit; ++i)
    w[i >> 2] |= ((fabsf(v[i]) < INFINITY ? 0u : 0x7Fu) | sign80(i)) << (8 * (i & 3));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// One 8-bit output with its scales, row-major; the format is uniform over a launch.
struct Fp8Out {
  uint8_t* codes;   // [rows, cols]
  void* scales;     // FP32 [rows, ceil(cols / 128)] or, with mx, UE8M0 [rows, cols / 32]
  int32_t per_row;  // scales per row
  bool e5m2, mx;
};

// Casts a unit and stores its codes and its block's scale.  All 32 lanes of a
// warp call this; the 8 lanes of a tile hold consecutive units of one row, and
// a lane past the row's end holds zeros and stores nothing (in_row false).
//
// 1x128 tiles follow fp8_quantize_blockwise: scale = amax / fp8_max, elements
// times r = fp8_max / amax, r = 0 for a tile of zeros or with a non-finite
// element.  A tile with 0 < amax < fp8_max / FLT_MAX would need a multiplier
// beyond binary32; it is cast with r = 0 too, so its elements (below 2^-112)
// become zeros instead of the NaN that 0 * inf would give.
// 1x32 blocks follow mx_quantize: e = max(floor(log2 amax) - emax, -127), scale
// byte e + 127, elements times 2^-e; a non-finite block has byte 0xFF, codes 0.
template <typename SignOf>
__device__ __forceinline__ void cast_store(const float (&v)[kUnit], const Fp8Out& o, int64_t row, int cols, int u,
                                           bool in_row, SignOf sign80) {
  uint32_t m = unit_amax(v);
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
  float mul, scale = 0.0f;
  uint32_t byte = 0u;
  if (o.mx) {
    const uint32_t E = m >> 23, emax = o.e5m2 ? 15u : 8u;
    byte = m >= 0x7F800000u ? 0xFFu : (E > emax ? E - emax : 0u);
    mul = m >= 0x7F800000u ? 0.0f : __uint_as_float((254u - byte) << 23);
  } else {
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 4));
    const float amax = __uint_as_float(m), top = o.e5m2 ? 57344.0f : 448.0f;
    scale = __fdiv_rn(amax, top);
    mul = __fdiv_rn(top, amax);
    if (!(mul < INFINITY) || m >= 0x7F800000u) mul = 0.0f;
  }
  uint4 c;
  if (__builtin_expect(m >= 0x7F800000u, 0))
    c = o.mx ? make_uint4(0u, 0u, 0u, 0u) : nonfinite_unit(v, sign80);
  else
    c = o.e5m2 ? cast_unit<true>(v, mul) : cast_unit<false>(v, mul);
  if (!in_row) return;
  st_cs(o.codes + row * cols + u * kUnit, c);
  if (o.mx) {
    if ((u & 1) == 0) static_cast<uint8_t*>(o.scales)[row * o.per_row + (u >> 1)] = (uint8_t)byte;
  } else {
    if ((u & 7) == 0)
      static_cast<float*>(o.scales)[row * o.per_row + (u >> 3)] = m > 0x7F800000u ? __uint_as_float(0x7FC00000u) : scale;
  }
}

// cast_store of computed values: a NaN's sign is the value's own.
__device__ __forceinline__ void cast_store(const float (&v)[kUnit], const Fp8Out& o, int64_t row, int cols, int u,
                                           bool in_row) {
  cast_store(v, o, row, cols, u, in_row, [&](int i) { return (__float_as_uint(v[i]) >> 24) & 0x80u; });
}

// Values of the 16 E4M3 codes of a unit times their tile's scale.
__device__ __forceinline__ void e4m3_floats(uint4 c, float scale, float (&f)[kUnit]) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const unsigned short two = (unsigned short)(w[k >> 1] >> (16 * (k & 1)));
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(two));
    f[2 * k] = __fmul_rn(f16lo(h2), scale);
    f[2 * k + 1] = __fmul_rn(f16hi(h2), scale);
  }
}

// Sum of one value per thread over the CTA's warps, in a fixed order, in every
// thread.  `slot` (32 floats) must not be rewritten before every thread has
// passed the next barrier: callers alternate between two.
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  return v;
}
__device__ __forceinline__ float block_sum(float v, float* slot) {
  v = warp_sum(v);
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) slot[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum(lane < warps ? slot[lane] : 0.0f);
}

}  // namespace mp
