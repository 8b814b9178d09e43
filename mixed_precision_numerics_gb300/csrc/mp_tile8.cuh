// mp_tile8.cuh — device building blocks of the block operators that read and
// write 8-bit tensors with scales (mp_norm.cu, mp_swiglu.cu).
//
// The unit of work is 16 consecutive elements of a row in one thread: 32 bytes
// of 16-bit input in two 16-byte loads, and exactly one 16-byte store of FP8
// codes.  A 1x128 tile is then eight lanes and a 1x32 block two, so a tile
// maximum takes three shuffles (one for 1x32) and no shared memory.
//
// With three 8-bit outputs a unit costs some 400 instructions, about what the
// SMs issue in the time its bytes take (2.4 of 4 a cycle), so the arithmetic is
// kept short: element pairs go through the packed binary32 instructions (each
// half rounded as the scalar one would), the stream's sum through the packed
// 16-bit addition, and all divisions of a tile are one, a lane each.  That took
// the norm of [8192 x 4096] BF16 with its checkpoint from 647 to 366
// instructions a unit and from 56.5 to 42.8 us.
#pragma once

#include "mp_device.cuh"

namespace mp {

enum { XF32 = 0, XF16 = 1, XBF16 = 2 };  // the values of mp_dtype

constexpr int kUnit = 16;               // elements per unit
constexpr int kPairs = kUnit / 2;
constexpr int kTile = 128;              // elements per FP32 scale
constexpr int kTileLanes = kTile / kUnit;

// ---------------------------------------------------------------------------
// Packed binary32 pairs.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint64_t pack64(float2 a) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
  return r;
}
__device__ __forceinline__ float2 unpack64(uint64_t a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pack64(a)), "l"(pack64(b)));
  return unpack64(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pack64(a)), "l"(pack64(b)));
  return unpack64(r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(pack64(a)), "l"(pack64(b)), "l"(pack64(c)));
  return unpack64(r);
}
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

// NaN-propagating max(|a|, |b|, |c|).
__device__ __forceinline__ float max3_abs_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// 32-bit division by a launch constant: n / d = floor(n * mul / 2^(31 + shift))
// for n < 2^31, mul = ceil(2^(31 + shift) / d) (the round-up reciprocal of
// Granlund and Montgomery, PLDI'94).
struct FastDiv {
  uint32_t d, mul, shift;
};
inline FastDiv fast_div(uint32_t d) {
  FastDiv f{d, 0u, 0u};
  while ((1ull << f.shift) < d) ++f.shift;  // 2^shift >= d
  f.mul = (uint32_t)(((1ull << (31 + f.shift)) + d - 1) / d);  // below 2^32, as 2^shift < 2d
  return f;
}
__device__ __forceinline__ uint32_t div_by(uint32_t n, const FastDiv& f) {
  return (uint32_t)(((uint64_t)n * f.mul) >> 31) >> f.shift;
}

// 16 or 8 bytes of shared memory, read where this is written and not kept.
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "r"(addr)
               : "memory");
  return r;
}
__device__ __forceinline__ uint2 lds8(uint32_t addr) {
  uint2 r;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(addr) : "memory");
  return r;
}

// ---------------------------------------------------------------------------
// One unit as loaded: 16 elements of type XT.
// ---------------------------------------------------------------------------
template <int XT>
struct Unit {
  static constexpr int kBytes = kUnit * (XT == XF32 ? 4 : 2);
  static constexpr int kVecs = kBytes / 16;
  uint4 v[kVecs];

  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) v[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  // the unit at element `at` of `base`
  __device__ __forceinline__ void load(const void* base, int64_t at) {
    const unsigned char* p = static_cast<const unsigned char*>(base) + at * (kBytes / kUnit);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) v[i] = ld_cs(p + 16 * i);
  }
  __device__ __forceinline__ void store(void* base, int64_t at) const {
    unsigned char* p = static_cast<unsigned char*>(base) + at * (kBytes / kUnit);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) st_cs(p + 16 * i, v[i]);
  }
  // A unit in halves of 8 elements: half `half` of this from an address of
  // shared or global memory.
  __device__ __forceinline__ void take_half(uint32_t addr, int half) {
#pragma unroll
    for (int i = 0; i < kVecs / 2; ++i) v[half * (kVecs / 2) + i] = lds16(addr + 16 * i);
  }
  __device__ __forceinline__ void load_half(const char* p, int half) {
#pragma unroll
    for (int i = 0; i < kVecs / 2; ++i) v[half * (kVecs / 2) + i] = ld_cs(p + 16 * i);
  }
  __device__ __forceinline__ void store_half(char* p, int half) const {
#pragma unroll
    for (int i = 0; i < kVecs / 2; ++i) st_cs(p + 16 * i, v[half * (kVecs / 2) + i]);
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
  __device__ __forceinline__ void floats(float2 (&f)[kPairs]) const {
#pragma unroll
    for (int k = 0; k < kPairs; ++k) f[k] = pair(k);
  }
  // Rounds a pair to XT, to nearest even.  The conversion gives 0x7FFF for
  // every NaN, as pack_f16x2 / pack_bf16x2 do.
  __device__ __forceinline__ void set_pair(int k, float2 a) {
    if constexpr (XT == XF32) {
      set_word(2 * k, __float_as_uint(a.x));
      set_word(2 * k + 1, __float_as_uint(a.y));
    } else {
      uint32_t r;
      if constexpr (XT == XF16)
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(a.y), "f"(a.x));
      else
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(a.y), "f"(a.x));
      set_word(k, r);
    }
  }
  // Adds another unit, each sum rounded to XT.  For the 16-bit types one
  // packed addition rounds once; rounding the binary32 sum gives the same
  // value, as 24 bits are at least 2 * 11 + 2.
  __device__ __forceinline__ void add(const Unit& o) {
    if constexpr (XT == XF32) {
#pragma unroll
      for (int k = 0; k < kPairs; ++k) set_pair(k, add2(pair(k), o.pair(k)));
    } else {
#pragma unroll
      for (int k = 0; k < kPairs; ++k) {
        uint32_t r;
        if constexpr (XT == XF16)
          asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(word(k)), "r"(o.word(k)));
        else
          asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(word(k)), "r"(o.word(k)));
        set_word(k, r);
      }
    }
  }
  // Makes the compiler unpack the words again from here on, instead of keeping
  // an earlier use's 16 floats in registers.
  __device__ __forceinline__ void forget() {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) asm volatile("" : "+r"(v[i].x), "+r"(v[i].y), "+r"(v[i].z), "+r"(v[i].w));
  }
  // the sign bit of element i as stored (a conversion may drop a NaN's sign)
  __device__ __forceinline__ uint32_t sign80(int i) const {
    if constexpr (XT == XF32) return (word(i) >> 24) & 0x80u;
    return (word(i >> 1) >> ((i & 1) ? 24 : 8)) & 0x80u;
  }
};

// 16 weights of a vector of any of the three types (a uniform branch), as
// stored.  The vector is read again for every row: default caching keeps it in
// L1.  The loads are volatile so that they stay where they are written, early
// to be in flight or late to be in registers only while they are used, and not
// through the read-only path: the kernel before, which may have written the
// weights, can still run when this one is launched.
struct Weights {
  uint4 v[4];
  __device__ __forceinline__ static uint4 load16(const uint4* p) {
    uint4 r;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p)
                 : "memory");
    return r;
  }
  __device__ __forceinline__ void load(const void* w, int wt, int u) {
    const uint4* p = static_cast<const uint4*>(w) + u * (wt == XF32 ? 4 : 2);
    v[0] = load16(p), v[1] = load16(p + 1);
    if (wt == XF32) v[2] = load16(p + 2), v[3] = load16(p + 3);
  }
  __device__ __forceinline__ void floats(int wt, float2 (&f)[kPairs]) const {
    if (wt == XF32) {
      Unit<XF32> r;
#pragma unroll
      for (int i = 0; i < 4; ++i) r.v[i] = v[i];
      r.floats(f);
    } else if (wt == XBF16) {
      Unit<XBF16> r;
      r.v[0] = v[0], r.v[1] = v[1];
      r.floats(f);
    } else {
      Unit<XF16> r;
      r.v[0] = v[0], r.v[1] = v[1];
      r.floats(f);
    }
  }
};

// NaN-propagating max |v| of a unit, as bits that order as integers: the NaN
// that the instruction gives is positive and above infinity.
__device__ __forceinline__ uint32_t unit_amax(const float2 (&v)[kPairs]) {
  float a = 0.0f, b = 0.0f;
#pragma unroll
  for (int k = 0; k < kPairs; k += 2) {
    a = max3_abs_nan(a, v[k].x, v[k].y);
    b = max3_abs_nan(b, v[k + 1].x, v[k + 1].y);
  }
  return __float_as_uint(max3_abs_nan(a, b, b));
}
// Maximum over the 8 lanes of a tile, or the 2 of a 1x32 block.
__device__ __forceinline__ uint32_t pair_max(uint32_t m) { return max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1)); }
__device__ __forceinline__ uint32_t tile_max(uint32_t m) {
  m = pair_max(m);
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
  return max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 4));
}

constexpr uint32_t kInfBits = 0x7F800000u;

// Multipliers and stored scales of the first M of N 1x128 tiles at once (the
// same eight lanes hold them all), by fp8_quantize_blockwise's rule: scale =
// amax / top, multiplier top / amax, with `top` for tile N - 1 (the output) and
// 448 for the others (checkpoints).  Both are correctly rounded divisions; lane
// 2k of the tile's eight does tile k's multiplier and lane 2k + 1 its scale, so
// one division serves them all.  mul[k] is valid in every lane, *scale in lane
// 2k + 1.  The multiplier is 0 for a tile of zeros, with a non-finite element,
// or with an amax below top / FLT_MAX (2^-119 in E4M3, 2^-112 in E5M2), where top /
// amax would be infinite: its elements become zeros instead of the NaN that 0 * inf would give.
template <int N, int M>
__device__ __forceinline__ void tile_scales(const uint32_t (&m)[N], float top, float (&mul)[N], float* scale) {
  const int lane = threadIdx.x & 7;
  uint32_t mm = m[0];
#pragma unroll
  for (int k = 1; k < M; ++k) mm = lane >= 2 * k ? m[k] : mm;
  const float tt = M == N && lane >= 2 * (N - 1) ? top : 448.0f;
  const float amax = __uint_as_float(mm);
  const float q = __fdiv_rn((lane & 1) ? amax : tt, (lane & 1) ? tt : amax);
  const float r = (q < INFINITY && mm < kInfBits) ? q : 0.0f;
#pragma unroll
  for (int k = 0; k < M; ++k) mul[k] = __shfl_sync(0xFFFFFFFFu, r, (threadIdx.x & 24) + 2 * k);
  *scale = mm > kInfBits ? __uint_as_float(0x7FC00000u) : q;
}
// The same of a 1x32 block by mx_quantize's rule: e = max(floor(log2 amax) -
// emax, -127), byte e + 127, multiplier 2^-e; byte 0xFF for a non-finite one.
__device__ __forceinline__ void mx_scale(uint32_t m, uint32_t emax, float* mul, uint32_t* byte) {
  const uint32_t E = m >> 23, b = E > emax ? E - emax : 0u;
  *byte = m >= kInfBits ? 0xFFu : b;
  *mul = __uint_as_float((254u - b) << 23);
}

// Saturating codes of a unit whose products with `mul` are not NaN.
template <bool E5M2>
__device__ __forceinline__ uint4 cast_unit(const float2 (&v)[kPairs], float mul) {
  const float2 m = both(mul);
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 a = mul2(v[2 * k], m), b = mul2(v[2 * k + 1], m);
    w[k] = E5M2 ? cvt_e5m2x2(a.x, a.y) | (cvt_e5m2x2(b.x, b.y) << 16)
                : cvt_e4m3x2(a.x, a.y) | (cvt_e4m3x2(b.x, b.y) << 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Codes of a unit in a tile that holds an infinity or a NaN: 0x7F with the
// element's sign for each of those, a zero with its sign for a finite element.
template <typename SignOf>
__device__ __forceinline__ uint4 nonfinite_unit(const float2 (&v)[kPairs], SignOf sign80) {
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < kUnit; ++i) {
    const float f = (i & 1) ? v[i >> 1].y : v[i >> 1].x;
    w[i >> 2] |= ((fabsf(f) < INFINITY ? 0u : 0x7Fu) | sign80(i)) << (8 * (i & 3));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// One 8-bit output with its scales, row-major; the format is uniform over a launch.
struct Fp8Out {
  uint8_t* codes;   // [rows, cols]
  void* scales;     // FP32 [rows, ceil(cols / 128)] or, with mx, UE8M0 [rows, cols / 32]
  int32_t per_row;  // scales per row
  bool e5m2, mx;
};

// Place of a unit: element `at` = row * cols + u * 16 of a dense tensor.
struct Place {
  int64_t at;
  int32_t row, u;
  bool in;        // the unit lies in the tensor
  bool tile_in;   // its tile's first unit does
};

// Codes of 16 values of a tile or block whose maximum is m, stored if in range.
template <typename SignOf>
__device__ __forceinline__ void store_codes(const float2 (&v)[kPairs], uint8_t* codes, const Place& p, uint32_t m,
                                            float mul, bool e5m2, bool mx, SignOf sign80) {
  uint4 c;
  if (__builtin_expect(m >= kInfBits, 0))
    c = mx ? make_uint4(0u, 0u, 0u, 0u) : nonfinite_unit(v, sign80);
  else
    c = e5m2 ? cast_unit<true>(v, mul) : cast_unit<false>(v, mul);
  if (p.in) st_cs(codes + p.at, c);
}
// The sign of a computed value is the value's own, a NaN's too.
__device__ __forceinline__ uint32_t float_sign80(const float2 (&v)[kPairs], int i) {
  return (__float_as_uint((i & 1) ? v[i >> 1].y : v[i >> 1].x) >> 24) & 0x80u;
}

// Casts a unit's values y and stores codes and scale, and with N > 1 the N - 1
// checkpoints of tensors whose tiles have maxima mc (raw holds their elements
// as stored; codes in cc, scales in cs, `tiles` a row).  All 32 lanes of a
// warp call this; the 8 lanes of a tile hold consecutive units of one row.  A
// lane past the row's end may hold anything: `in` keeps it out of the maxima
// (the caller's mc too) and of the stores.
template <int N, int XT>
__device__ __forceinline__ void cast_store(const float2 (&y)[kPairs], const Fp8Out& o, const Place& p,
                                           const uint32_t (&mc)[N], Unit<XT> (&raw)[N], uint8_t* const (&cc)[N],
                                           float* const (&cs)[N], int tiles) {
  const int lane = threadIdx.x & 7;
  uint32_t my = pair_max(p.in ? unit_amax(y) : 0u);
  float mul[N], scale, mul_y;
  if (o.mx) {
    uint32_t byte;
    mx_scale(my, o.e5m2 ? 15u : 8u, &mul_y, &byte);
    if ((lane & 1) == 0 && p.in)
      static_cast<uint8_t*>(o.scales)[(int64_t)p.row * o.per_row + (p.u >> 1)] = (uint8_t)byte;
    if constexpr (N > 1) tile_scales<N, N - 1>(mc, 448.0f, mul, &scale);
  } else {
    my = max(my, __shfl_xor_sync(0xFFFFFFFFu, my, 2));
    my = max(my, __shfl_xor_sync(0xFFFFFFFFu, my, 4));
    uint32_t m[N];
#pragma unroll
    for (int k = 0; k < N - 1; ++k) m[k] = mc[k];
    m[N - 1] = my;
    tile_scales<N, N>(m, o.e5m2 ? 57344.0f : 448.0f, mul, &scale);
    mul_y = mul[N - 1];
    if (lane == 2 * N - 1 && p.tile_in) static_cast<float*>(o.scales)[(int64_t)p.row * o.per_row + (p.u >> 3)] = scale;
  }
  store_codes(y, o.codes, p, my, mul_y, o.e5m2, o.mx, [&](int i) { return float_sign80(y, i); });
#pragma unroll
  for (int k = 0; k < N - 1; ++k) {
    if (lane == 2 * k + 1 && p.tile_in) cs[k][(int64_t)p.row * tiles + (p.u >> 3)] = scale;
    float2 v[kPairs];
    raw[k].forget();
    raw[k].floats(v);
    store_codes(v, cc[k], p, mc[k], mul[k], false, false, [&](int i) { return raw[k].sign80(i); });
  }
}

// Without checkpoints.
template <int XT>
__device__ __forceinline__ void cast_store(const float2 (&y)[kPairs], const Fp8Out& o, const Place& p) {
  const uint32_t mc[1] = {0u};
  Unit<XT> raw[1];
  uint8_t* const cc[1] = {nullptr};
  float* const cs[1] = {nullptr};
  cast_store<1, XT>(y, o, p, mc, raw, cc, cs, 0);
}

// Values of the two E4M3 codes in the low (k even) or high half of a word,
// exact (through binary16).  Volatile: a second use converts the codes again
// instead of keeping 16 floats in registers.
__device__ __forceinline__ float2 e4m3_floats(uint32_t w, int k) {
  uint32_t h;
  asm volatile("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)(w >> (16 * (k & 1)))));
  return make_float2(f16lo(h), f16hi(h));
}

}  // namespace mp
