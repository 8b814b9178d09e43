// mp_swiglu.cu — the gated product of a feed-forward block with an FP8 output,
// and its backward pass from gate and up or from their 8-bit checkpoint.
//
// Forward: p = (g * s(g)) * u with s the logistic function; y = p in FP8 with
// one scale per 1x128 tile (FP32) or 1x32 block (UE8M0); optionally g and u in
// E4M3 with 1x128 scales, the checkpoint.
// Backward, with g and u as given or the checkpoint's values:
//   du = dp * (g * s(g)),  dg = dp * u * (s(g) * (1 + g * (1 - s(g)))).
//
// One thread owns 16 elements end to end, with every CTA launched at once;
// every element is read and written once.  gate and up (dgate and dup) may be
// column ranges of one wider matrix: each pair has a row distance.
//
// Bound by DRAM.  [8192 x 14336] BF16 forward with the checkpoint, 7.1 bytes an
// element and 400 instructions for 16: 124.0 us, 0.99 of the copy rate (6793
// GB/s); backward from the checkpoint, 8.1 bytes: 135.8 us, 1.03; from gate and
// up, 10 bytes: [2048 x 12288] 38.8 us, 0.95.  What counts is how many units are
// on an SM: CTAs of 128 threads, nine of them (56 registers) forward and twelve
// (40, which spill 20 to 24 bytes a thread) backward for the 16-bit types.  (256
// threads, four and six CTAs: 132.9 and 138.9 us; 512 threads: 137.5 and 142.5; 36
// registers backward, which spill more: 147.6.  The forward tile's three pairs of
// divisions one by one: 157.)
//
// FP32 [8192 x 8192], us by CTAs an SM: forward, with the checkpoint and without,
// four 111.7 and 90.6, six 107.5 and 86.4, seven 106.1 and 85.4, nine 110.8 and 85.5;
// backward from the checkpoint four 158.7, six 152.3, seven 148.6, ten 155.0; from
// gate and up, more bytes of which are in flight a thread, four 185.8, six 188.6,
// seven 190.1.
#include "mp_chain.cuh"
#include "mp_internal.h"
#include "mp_tile8.cuh"

namespace mp {
namespace {

constexpr int kThreads = 128;

// Thread q holds lane q % 8 of tile q / 8; tiles run along rows.
__device__ __forceinline__ Place place_of(int64_t rows, int cols, const FastDiv& tiles) {
  const uint32_t tile = blockIdx.x * (kThreads / kTileLanes) + threadIdx.x / kTileLanes;  // below 2^31
  Place p;
  p.row = (int32_t)div_by(tile, tiles);
  p.u = (int32_t)((tile - p.row * tiles.d) * kTileLanes + threadIdx.x % kTileLanes);
  p.tile_in = p.row < rows;
  p.in = p.tile_in && p.u * kUnit < cols;
  p.at = (int64_t)p.row * cols + p.u * kUnit;
  return p;
}

struct SwigluFwd {
  const void *gate, *up;
  int64_t ld;  // elements between rows of gate, and of up
  Fp8Out y;
  uint8_t* ckpt;  // gate's, then up's; NULL for none
  float* ckpt_scales;
  int64_t rows;
  int32_t cols;
  FastDiv tiles;
};

template <int XT, bool SAVE>
__global__ __launch_bounds__(kThreads, XT == XF32 ? 7 : 9) void k_swiglu_fwd(const __grid_constant__ SwigluFwd a) {
  chain_wait();
  chain_release();
  constexpr int N = SAVE ? 3 : 1;
  const Place p = place_of(a.rows, a.cols, a.tiles);
  Unit<XT> raw[3];
  raw[0].zero();
  raw[1].zero();
  if (p.in) {
    const int64_t at = p.row * a.ld + p.u * kUnit;
    raw[0].load(a.gate, at);
    raw[1].load(a.up, at);
  }
  float2 y[kPairs];
  float ag = 0.0f, au = 0.0f;
#pragma unroll
  for (int k = 0; k < kPairs; ++k) {
    const float2 g = raw[0].pair(k), u = raw[1].pair(k);
    if constexpr (SAVE) {
      ag = max3_abs_nan(ag, g.x, g.y);
      au = max3_abs_nan(au, u.x, u.y);
    }
    y[k] = mul2(mul2(g, logistic2<XT>(g)), u);
  }
  if constexpr (SAVE) {
    const uint32_t mc[N] = {tile_max(__float_as_uint(ag)), tile_max(__float_as_uint(au)), 0u};
    uint8_t* const cc[N] = {a.ckpt, a.ckpt + a.rows * a.cols, nullptr};
    float* const cs[N] = {a.ckpt_scales, a.ckpt_scales + a.rows * a.tiles.d, nullptr};
    cast_store<N, XT>(y, a.y, p, mc, raw, cc, cs, a.tiles.d);
  } else {
    cast_store<XT>(y, a.y, p);
  }
}

struct SwigluBwd {
  const void *dp, *gate, *up;
  const uint8_t* codes;  // the 8-bit checkpoint [2][rows][cols], or NULL where gate and up are given
  const float* scales;   // [2][rows][tiles]
  void *dgate, *dup;
  int64_t ld, d_ld, rows;  // elements between rows of gate and up, of dgate and dup
  int32_t cols;
  FastDiv tiles;
};

template <int XT, bool SAVED>
__global__ __launch_bounds__(kThreads, XT != XF32 ? 12 : SAVED ? 7 : 4) void k_swiglu_bwd(const __grid_constant__ SwigluBwd a) {
  chain_wait();
  chain_release();
  const Place p = place_of(a.rows, a.cols, a.tiles);
  if (!p.in) return;
  Unit<XT> dr;
  float2 g[kPairs], u[kPairs];
  if constexpr (SAVED) {
    const int64_t st = (int64_t)p.row * a.tiles.d + p.u / kTileLanes;
    const uint4 gc = ld_cs(a.codes + p.at), uc = ld_cs(a.codes + a.rows * a.cols + p.at);
    const float gs = __ldcs(a.scales + st), us = __ldcs(a.scales + a.rows * a.tiles.d + st);
    dr.load(a.dp, p.at);
    const uint32_t gw[4] = {gc.x, gc.y, gc.z, gc.w}, uw[4] = {uc.x, uc.y, uc.z, uc.w};
#pragma unroll
    for (int k = 0; k < kPairs; ++k) {
      g[k] = mul2(e4m3_floats(gw[k >> 1], k), both(gs));
      u[k] = mul2(e4m3_floats(uw[k >> 1], k), both(us));
    }
  } else {
    Unit<XT> gr, ur;
    const int64_t at = p.row * a.ld + p.u * kUnit;
    gr.load(a.gate, at);
    ur.load(a.up, at);
    dr.load(a.dp, p.at);
    gr.floats(g);
    ur.floats(u);
  }
  Unit<XT> dg, du;
#pragma unroll
  for (int k = 0; k < kPairs; ++k) {
    const float2 d = dr.pair(k), s = logistic2<XT>(g[k]), xs = mul2(g[k], s);
    du.set_pair(k, mul2(d, xs));
    const float2 one_s = fma2(s, both(-1.0f), both(1.0f));
    dg.set_pair(k, mul2(mul2(d, u[k]), fma2(xs, one_s, s)));
  }
  const int64_t at = p.row * a.d_ld + p.u * kUnit;
  dg.store(a.dgate, at);
  du.store(a.dup, at);
}

unsigned ctas_of(int64_t rows, const FastDiv& tiles) {
  return (unsigned)((rows * tiles.d * kTileLanes + kThreads - 1) / kThreads);
}

template <int XT>
mp_status launch_fwd(const SwigluFwd& a, cudaStream_t st) {
  const dim3 g(ctas_of(a.rows, a.tiles)), b(kThreads);
  if (a.ckpt)
    launch_chained(k_swiglu_fwd<XT, true>, g, b, 0, st, a);
  else
    launch_chained(k_swiglu_fwd<XT, false>, g, b, 0, st, a);
  note_launches(1);
  return launch_status();
}
template <int XT>
mp_status launch_bwd(const SwigluBwd& a, cudaStream_t st) {
  const dim3 g(ctas_of(a.rows, a.tiles)), b(kThreads);
  if (a.codes)
    launch_chained(k_swiglu_bwd<XT, true>, g, b, 0, st, a);
  else
    launch_chained(k_swiglu_bwd<XT, false>, g, b, 0, st, a);
  note_launches(1);
  return launch_status();
}

bool float_type(mp_dtype t) { return t == MP_F32 || t == MP_F16 || t == MP_BF16; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Whether a matrix of `cols` columns may have rows `ld` elements apart: they
// must not overlap, and each has to start on 16 bytes.  Byte offsets are 64-bit.
bool pitch_ok(int64_t ld, int64_t cols, int64_t rows, mp_dtype t) {
  return rows <= 1 || (ld >= cols && ld < (1ll << 61) / rows && ld % (t == MP_F32 ? 4 : 8) == 0);
}
// Tile numbers (2.7e11 elements: more than the device's memory holds of any
// input), rows and the columns up to the end of a row's last tile are 32-bit.
bool shape_ok(int64_t rows, int64_t cols, int step) {
  if (rows >= (1ll << 31) || cols > (1ll << 31) - kTile || cols % step != 0) return false;
  return rows * ((cols + kTile - 1) / kTile) < (1ll << 31) - kThreads / kTileLanes;
}

}  // namespace
}  // namespace mp

extern "C" MP_API mp_status swiglu_fp8(const void* gate, const void* up, int64_t ld, mp_dtype x_dtype, int64_t rows,
                                       int64_t cols, void* y, mp_dtype fp8_dtype, int32_t scale_block, void* y_scales,
                                       void* ckpt, float* ckpt_scales, void* stream) {
  using namespace mp;
  if (rows < 0 || cols < 0) return MP_EINVAL;
  if (!float_type(x_dtype)) return MP_EINVAL;
  if (fp8_dtype != MP_E4M3 && fp8_dtype != MP_E5M2) return MP_EINVAL;
  if (scale_block != 128 && scale_block != 32) return MP_EINVAL;
  if (!shape_ok(rows, cols, scale_block == 32 ? 32 : 16)) return MP_ESHAPE;
  if (rows == 0 || cols == 0) return MP_OK;
  if (!gate || !up || !y || !y_scales || (!ckpt != !ckpt_scales)) return MP_EINVAL;
  if (!pitch_ok(ld, cols, rows, x_dtype)) return MP_ESHAPE;
  if (!aligned16(gate) || !aligned16(up) || !aligned16(y) || !aligned16(ckpt) || !aligned4(ckpt_scales) ||
      (scale_block == 128 && !aligned4(y_scales)))
    return MP_EALIGN;
  SwigluFwd a;
  const int32_t tiles = (int32_t)((cols + kTile - 1) / kTile);
  a.gate = gate, a.up = up, a.ld = ld, a.rows = rows, a.cols = (int32_t)cols, a.tiles = fast_div(tiles);
  a.y = Fp8Out{static_cast<uint8_t*>(y), y_scales, scale_block == 32 ? (int32_t)(cols / 32) : tiles,
               fp8_dtype == MP_E5M2, scale_block == 32};
  a.ckpt = static_cast<uint8_t*>(ckpt), a.ckpt_scales = ckpt_scales;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (x_dtype) {
    case MP_F32: return launch_fwd<XF32>(a, st);
    case MP_F16: return launch_fwd<XF16>(a, st);
    default: return launch_fwd<XBF16>(a, st);
  }
}

extern "C" MP_API mp_status swiglu_backward(const void* dp, mp_dtype x_dtype, int64_t rows, int64_t cols,
                                            const void* gate, const void* up, int64_t ld, const void* ckpt,
                                            const float* ckpt_scales, void* dgate, void* dup, int64_t d_ld,
                                            void* stream) {
  using namespace mp;
  if (rows < 0 || cols < 0) return MP_EINVAL;
  if (!float_type(x_dtype)) return MP_EINVAL;
  if (!shape_ok(rows, cols, 16)) return MP_ESHAPE;
  if (rows == 0 || cols == 0) return MP_OK;
  if (!dp || !dgate || !dup || (!ckpt != !ckpt_scales) || (!gate != !up) || (!gate == !ckpt)) return MP_EINVAL;
  if ((gate && !pitch_ok(ld, cols, rows, x_dtype)) || !pitch_ok(d_ld, cols, rows, x_dtype)) return MP_ESHAPE;
  if (!aligned16(dp) || !aligned16(gate) || !aligned16(up) || !aligned16(ckpt) || !aligned4(ckpt_scales) ||
      !aligned16(dgate) || !aligned16(dup))
    return MP_EALIGN;
  SwigluBwd a;
  a.dp = dp, a.gate = gate, a.up = up, a.codes = static_cast<const uint8_t*>(ckpt), a.scales = ckpt_scales;
  a.dgate = dgate, a.dup = dup, a.ld = ld, a.d_ld = d_ld, a.rows = rows, a.cols = (int32_t)cols;
  a.tiles = fast_div((uint32_t)((cols + kTile - 1) / kTile));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (x_dtype) {
    case MP_F32: return launch_bwd<XF32>(a, st);
    case MP_F16: return launch_bwd<XF16>(a, st);
    default: return launch_bwd<XBF16>(a, st);
  }
}
