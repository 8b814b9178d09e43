// mp_ffn.cuh — what the two kernels of the gated feed-forward products share:
// mp_ffn.cu for many rows, mp_ffn_few.cu for up to kFewRows.
#pragma once

#include "mp_internal.h"
#include "mp_mma.cuh"
#include "mp_tile8.cuh"

namespace mp {

// What becomes of a product.
enum {
  FWD16 = 0,  // p in 16 bits
  FWD8,       // p in FP8
  AGAIN,      // g and u formed again: dg and du
  STORE       // the product itself
};

constexpr int kBlockK = 64;    // steps of the contraction in a stage: 128 bytes
// Up to kFewDxRows rows the products have the kernel of few rows, the forward
// product up to kFewRows where the weights are large, so that their way from DRAM
// counts most.  (Its time grows with the rows: 100 rows of 4096 x 14336 44.2 us, the
// other kernel's 129 rows 48.6; of 2048 x 5504 15.5 and 15.8, of 1024 x 2816 9.0 and
// 7.5.)
// dx of more rows shares the launch of the weights' gradients.  Its bits must not
// depend on whether those are asked for, so one rule serves both calls.  Up to 64
// rows a kernel of its own is much faster alone and not far off beside them (us by
// rows, of its own and in the shared launch, swiglu_backward included):
//                 dx alone             all gradients
//   4096 x 14336  1: 40, 70  64: 46, 70    1: 92, 97   64: 97, 100
//   2048 x 5504   1: 13, 24  64: 17, 25    1: 27, 28   64: 35, 31
//   1024 x 2816   1: 8, 13   64: 9, 13     1: 14, 13.5 64: 20, 19
//   256 x 688     1: 5, 9    64: 6.5, 9    1: 8.4, 8.9 64: 10.1, 9.3
// 100 rows of 2048 x 5504 with all gradients: 39.6 and 32.4.
constexpr int kFewRows = 128, kFewDxRows = 64;
constexpr int64_t kLargeWeights = 1 << 23;  // elements of each
inline bool few_forward(int64_t rows, int64_t width, int64_t hidden) {
  return rows <= kFewDxRows || (rows <= kFewRows && width * hidden >= kLargeWeights);
}

// Stages added up inside the tensor core, at most, before the sums move on to
// registers: 512 terms where FP32 scales show the truncation, those of an FP8
// product or of the 8-bit checkpoint (1024 would save 4 % of the time), 2048 where
// results are rounded to 16 bits.  Every instruction cuts off up to a step of a
// binary32 sum, so a run of T terms ends up to T / 16 * 2^-23 too small, relative.
constexpr int kShortRun = 8, kLongRun = 32;

template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float2 v) {  // a NaN gives 0x7FFF
  uint32_t r;
  if constexpr (BF16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(v.y), "f"(v.x));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(v.y), "f"(v.x));
  return r;
}
template <bool BF16>
__device__ __forceinline__ float2 pair16(uint32_t w) {
  return BF16 ? make_float2(bf16lo(w), bf16hi(w)) : make_float2(f16lo(w), f16hi(w));
}

// Scale and multiplier of a 1x128 tile by the rule of the other block operators
// (tile_scales), one thread for the tile.
__device__ __forceinline__ float tile_scale(uint32_t m, float top, float* mul) {
  const float amax = __uint_as_float(m), r = __fdiv_rn(top, amax);
  *mul = (r < INFINITY && m < kInfBits) ? r : 0.0f;
  return m > kInfBits ? __uint_as_float(0x7FC00000u) : __fdiv_rn(amax, top);
}

// p of a pair.
__device__ __forceinline__ float2 gated(float2 g, float2 u) { return mul2(mul2(g, logistic2<XF32>(g)), u); }
// dg and du of a pair.
__device__ __forceinline__ void slopes(float2 d, float2 g, float2 u, float2* dg, float2* du) {
  const float2 s = logistic2<XF32>(g), xs = mul2(g, s), one_s = fma2(s, both(-1.0f), both(1.0f));
  *dg = mul2(mul2(d, u), fma2(xs, one_s, s));
  *du = mul2(d, xs);
}

inline int32_t ceil_div(int64_t a, int64_t b) { return (int32_t)((a + b - 1) / b); }

// A matrix of 16-bit elements with rows `pitch` elements apart, in boxes of box_rows x 64.
inline bool map16(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, int64_t pitch, int box_rows) {
  return encode_swizzled_map_2d(m, p, rows, cols, pitch * 2, box_rows);
}

// What the forward call writes, and what AGAIN reads and writes.
struct FfnOut {
  void* p;         // FWD16: 16 bits; FWD8: codes
  bool e5m2, mx;
  void* p_scales;
  int32_t per_row, tiles;  // scales of p, and 1x128 tiles, in a row
  void *gate, *up;         // 16 bits, `ld` elements a row; or NULL
  int64_t ld;
  uint8_t* ckpt;           // [2][rows][hidden] or NULL
  float* ckpt_scales;      // [2][rows][tiles]
  const void* dp;          // AGAIN
  void *dg, *du;           // AGAIN: [rows][hidden] each
};

template <int EP>
__host__ __device__ __forceinline__ int run_of(const FfnOut& o) {
  return EP == FWD8 || (EP == FWD16 && o.ckpt) ? kShortRun : kLongRun;
}

// x [rows, width] and the weights [hidden, width]: FWD16, FWD8 or AGAIN for up to kFewRows rows.
mp_status ffn_few_project(int ep, bool bf16, const void* x, const void* w_gate, const void* w_up, int64_t rows,
                          int64_t width, int64_t hidden, const FfnOut& out, cudaStream_t st);
// dx = dg w_gate + du w_up for up to kFewDxRows rows.
mp_status ffn_few_dx(bool bf16, const void* dg, const void* du, const void* w_gate, const void* w_up, int64_t rows,
                     int64_t width, int64_t hidden, void* dx, cudaStream_t st);

uint32_t ffn_few_wait_failures();

}  // namespace mp
