// mp_norm.cu — root-mean-square norm with the residual's addition and an FP8
// output, and its backward pass from the stream or from its 8-bit checkpoint.
//
// Forward, per row of x and residual r (all of one type):
//   h = RNE(x + r), rstd = 1 / sqrt(mean(h^2) + eps), n = (h * rstd) * w,
//   y = n in FP8 with one scale per 1x128 tile (FP32) or 1x32 block (UE8M0),
//   and optionally h in E4M3 with 1x128 scales, the checkpoint.
// The norm is taken of the stored, rounded h: it is what the next block and
// the backward pass read, so the gradient is that of the function computed.
//
// Backward, with v = h or the checkpoint's values, xh = v * rstd, g = dy * w:
//   c = mean(g * xh),  dx = rstd * (g - xh * c) + dh,  dw = sum_rows dy * xh.
//
// Both read and write every element once: the row lives in registers between
// the two uses of it, before and after the row's sum.
#include <math.h>

#include "mp_chain.cuh"
#include "mp_internal.h"
#include "mp_tile8.cuh"

namespace mp {
namespace {

constexpr int kCta = 256;          // threads of a CTA that takes several rows
constexpr int kMaxThreads = 512;   // threads of a CTA that takes one row at a time
constexpr int kMaxUnits = 4;       // units of a row per thread
constexpr int kMaxCols = kMaxThreads * kMaxUnits * kUnit;
constexpr int kMaxParts = 608;     // partial sums of dweight: four CTAs on each of 152 SMs

// How a row is laid over threads, by its length alone.  `lanes` > 0: that many
// lanes of a warp hold the row and a CTA takes kCta / lanes rows; else a whole
// CTA of `threads` holds it, `units` 16-element units a thread.
struct RowShape {
  int lanes, threads, units, rows_per_cta;
};
RowShape row_shape(int64_t cols) {
  const int n = (int)(cols / kUnit);
  if (n <= 32) {
    const int l = n <= 8 ? 8 : n <= 16 ? 16 : 32;
    return {l, kCta, 1, kCta / l};
  }
  const int u = n <= kMaxThreads ? 1 : n <= 2 * kMaxThreads ? 2 : 4;
  const int t = ((n + u - 1) / u + 31) / 32 * 32;
  return {0, t, u, 1};
}

// Sum over the threads that hold one row, in every one of them.
template <int L>
__device__ __forceinline__ float row_sum(float v, float* slot) {
  if constexpr (L == 0) {
    return block_sum(v, slot);
  } else {
#pragma unroll
    for (int d = L / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    return v;
  }
}

// ---------------------------------------------------------------------------
// Forward
// ---------------------------------------------------------------------------
struct NormFwd {
  const void *x, *residual, *weight;
  void* h;
  float* rstd;
  Fp8Out y, ckpt;
  int64_t rows;
  int32_t cols, wt;
  float eps;
};

template <int XT, int L, int U>
__global__ __launch_bounds__(L ? kCta : kMaxThreads) void k_norm_fwd(const __grid_constant__ NormFwd a) {
  __shared__ float slots[2][32];
  chain_wait();
  chain_release();
  constexpr int R = L ? kCta / L : 1;
  const int t = L ? threadIdx.x % (L ? L : 1) : threadIdx.x, sub = L ? threadIdx.x / (L ? L : 1) : 0;
  const int stride = L ? L : blockDim.x, units = a.cols / kUnit;
  int parity = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * R; row0 < a.rows; row0 += (int64_t)gridDim.x * R, parity ^= 1) {
    const int64_t row = row0 + sub;
    Place p[U];
    Unit<XT> h[U];
    float2 ss = both(0.0f);
#pragma unroll
    for (int k = 0; k < U; ++k) {
      p[k].row = (int32_t)row;
      p[k].u = t + k * stride;
      p[k].at = row * a.cols + p[k].u * kUnit;
      p[k].in = row < a.rows && p[k].u < units;
      p[k].tile_in = row < a.rows && (p[k].u & ~7) < units;
      h[k].zero();
      if (p[k].in) {
        h[k].load(a.x, p[k].at);
        if (a.residual) {
          Unit<XT> r;
          r.load(a.residual, p[k].at);
          h[k].add(r);
        }
        if (a.h) h[k].store(a.h, p[k].at);
      }
      float2 f[kPairs];
      h[k].floats(f);
      if (a.ckpt.codes) cast_store(f, a.ckpt, p[k], [&](int i) { return h[k].sign80(i); });
#pragma unroll
      for (int i = 0; i < kPairs; ++i) ss = fma2(f[i], f[i], ss);
    }
    const float sum = row_sum<L>(ss.x + ss.y, slots[parity]);
    const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(sum, (float)a.cols), a.eps)));
    if (t == 0 && row < a.rows && a.rstd) a.rstd[row] = rstd;
#pragma unroll
    for (int k = 0; k < U; ++k) {
      float2 f[kPairs], w[kPairs];
#pragma unroll
      for (int i = 0; i < kPairs; ++i) f[i] = w[i] = both(0.0f);
      if (p[k].in) {
        h[k].floats(f);
        load_weights(a.weight, a.wt, p[k].u, w);
#pragma unroll
        for (int i = 0; i < kPairs; ++i) f[i] = mul2(mul2(f[i], both(rstd)), w[i]);
      }
      cast_store(f, a.y, p[k]);
    }
  }
}

template <int XT, int L, int U>
mp_status launch_fwd(const NormFwd& a, const RowShape& s, cudaStream_t st) {
  const int64_t ctas = (a.rows + s.rows_per_cta - 1) / s.rows_per_cta;
  launch_chained(k_norm_fwd<XT, L, U>, dim3(full_grid(ctas)), dim3(s.threads), 0, st, a);
  note_launches(1);
  return launch_status();
}

template <int XT>
mp_status launch_fwd_shape(const NormFwd& a, cudaStream_t st) {
  const RowShape s = row_shape(a.cols);
  if (s.lanes == 8) return launch_fwd<XT, 8, 1>(a, s, st);
  if (s.lanes == 16) return launch_fwd<XT, 16, 1>(a, s, st);
  if (s.lanes == 32) return launch_fwd<XT, 32, 1>(a, s, st);
  if (s.units == 1) return launch_fwd<XT, 0, 1>(a, s, st);
  if (s.units == 2) return launch_fwd<XT, 0, 2>(a, s, st);
  return launch_fwd<XT, 0, 4>(a, s, st);
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------
struct NormBwd {
  const void *dy, *dh, *h, *weight;
  const uint8_t* codes;  // the 8-bit checkpoint, or NULL where h is given
  const float *scales, *rstd;
  void* dx;
  float* parts;
  int64_t rows;
  int32_t cols, tiles, wt;
};

// CTA c takes row groups c, c + gridDim.x, ...; each thread keeps the sums of
// its own columns in registers over those rows (binary32, in row order) and
// the CTA writes one row of `parts` at the end.
template <int XT, bool SAVED, int L, int U>
__global__ __launch_bounds__(L ? kCta : kMaxThreads) void k_norm_bwd(const __grid_constant__ NormBwd a) {
  __shared__ float slots[2][32];
  __shared__ float fold[L ? kCta * kUnit : 1];
  chain_wait();
  chain_release();
  constexpr int R = L ? kCta / L : 1;
  const int t = L ? threadIdx.x % (L ? L : 1) : threadIdx.x, sub = L ? threadIdx.x / (L ? L : 1) : 0;
  const int stride = L ? L : blockDim.x, units = a.cols / kUnit;
  float2 acc[U][kPairs];
#pragma unroll
  for (int k = 0; k < U; ++k)
#pragma unroll
    for (int i = 0; i < kPairs; ++i) acc[k][i] = both(0.0f);
  int parity = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * R; row0 < a.rows; row0 += (int64_t)gridDim.x * R, parity ^= 1) {
    const int64_t row = row0 + sub;
    const bool live = row < a.rows;
    const float rstd = live ? a.rstd[row] : 0.0f;
    Unit<XT> dy[U], v[U];
    uint4 code[U];
    float scale[U];
    float2 dot = both(0.0f);
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int u = t + k * stride;
      const int64_t at = row * a.cols + u * kUnit;
      dy[k].zero();
      v[k].zero();
      code[k] = make_uint4(0u, 0u, 0u, 0u);
      scale[k] = 0.0f;
      if (live && u < units) {
        dy[k].load(a.dy, at);
        if constexpr (SAVED) {
          code[k] = ld_cs(a.codes + at);
          scale[k] = a.scales[row * a.tiles + u / kTileLanes];
        } else {
          v[k].load(a.h, at);
        }
      }
    }
    float2 g[U][kPairs], xh[U][kPairs];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int u = t + k * stride;
      if (live && u < units) {
        float2 w[kPairs];
        load_weights(a.weight, a.wt, u, w);
        if constexpr (SAVED) {
          e4m3_floats(code[k], scale[k] * rstd, xh[k]);
        } else {
          v[k].floats(xh[k]);
#pragma unroll
          for (int i = 0; i < kPairs; ++i) xh[k][i] = mul2(xh[k][i], both(rstd));
        }
        dy[k].floats(g[k]);
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          acc[k][i] = fma2(g[k][i], xh[k][i], acc[k][i]);
          g[k][i] = mul2(g[k][i], w[i]);
          dot = fma2(g[k][i], xh[k][i], dot);
        }
      }
    }
    const float c = __fdiv_rn(row_sum<L>(dot.x + dot.y, slots[parity]), (float)a.cols);
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int u = t + k * stride;
      if (live && u < units) {
        const int64_t at = row * a.cols + u * kUnit;
        Unit<XT> e, o;
        e.zero();
        if (a.dh) e.load(a.dh, at);
#pragma unroll
        for (int i = 0; i < kPairs; ++i)
          o.set_pair(i, fma2(fma2(xh[k][i], both(-c), g[k][i]), both(rstd), e.pair(i)));
        o.store(a.dx, at);
      }
    }
  }
  float* part = a.parts + (int64_t)blockIdx.x * a.cols;
  if constexpr (L == 0) {
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int u = t + k * stride;
      if (u < units) {
        float4* p = reinterpret_cast<float4*>(part + u * kUnit);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          p[i] = make_float4(acc[k][2 * i].x, acc[k][2 * i].y, acc[k][2 * i + 1].x, acc[k][2 * i + 1].y);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {  // [sub][t][element]
      fold[threadIdx.x * kUnit + 2 * i] = acc[0][i].x;
      fold[threadIdx.x * kUnit + 2 * i + 1] = acc[0][i].y;
    }
    __syncthreads();
    for (int col = threadIdx.x; col < a.cols; col += kCta) {
      float s = 0.0f;
      for (int j = 0; j < R; ++j) s += fold[j * (L * kUnit) + col];
      part[col] = s;
    }
  }
}

// dweight[col] = sum over the partial rows: 32 columns a CTA, 16 warps that
// each sum every 16th partial row, joined in a fixed order.
constexpr int kFoldWarps = 16;
__global__ __launch_bounds__(32 * kFoldWarps) void k_norm_dweight(const float* parts, int32_t nparts, int32_t cols,
                                                                  void* dweight, int32_t dt) {
  __shared__ float s[kFoldWarps][32];
  chain_wait();
  chain_release();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  float v = 0.0f;
  if (col < cols)
    for (int p = warp; p < nparts; p += kFoldWarps) v += parts[(int64_t)p * cols + col];
  s[warp][lane] = v;
  __syncthreads();
  if (warp != 0 || col >= cols) return;
  v = 0.0f;
#pragma unroll
  for (int j = 0; j < kFoldWarps; ++j) v += s[j][lane];
  if (dt == XF32)
    static_cast<float*>(dweight)[col] = v;
  else
    static_cast<uint16_t*>(dweight)[col] = (uint16_t)(dt == XF16 ? pack_f16x2(v, 0.0f) : pack_bf16x2(v, 0.0f));
}

int64_t parts_of(int64_t rows, int64_t cols) {
  const int64_t groups = (rows + row_shape(cols).rows_per_cta - 1) / row_shape(cols).rows_per_cta;
  return groups < kMaxParts ? groups : kMaxParts;
}

template <int XT, bool SAVED>
mp_status launch_bwd(const NormBwd& a, void* dweight, int32_t dt, cudaStream_t st) {
  const RowShape s = row_shape(a.cols);
  const int parts = (int)parts_of(a.rows, a.cols);
  if (parts > 0) {
    const dim3 g(parts), b(s.threads);
    if (s.lanes == 8)
      launch_chained(k_norm_bwd<XT, SAVED, 8, 1>, g, b, 0, st, a);
    else if (s.lanes == 16)
      launch_chained(k_norm_bwd<XT, SAVED, 16, 1>, g, b, 0, st, a);
    else if (s.lanes == 32)
      launch_chained(k_norm_bwd<XT, SAVED, 32, 1>, g, b, 0, st, a);
    else if (s.units == 1)
      launch_chained(k_norm_bwd<XT, SAVED, 0, 1>, g, b, 0, st, a);
    else if (s.units == 2)
      launch_chained(k_norm_bwd<XT, SAVED, 0, 2>, g, b, 0, st, a);
    else
      launch_chained(k_norm_bwd<XT, SAVED, 0, 4>, g, b, 0, st, a);
    note_launches(1);
  }
  launch_chained(k_norm_dweight, dim3((a.cols + 31) / 32), dim3(32 * kFoldWarps), 0, st, (const float*)a.parts,
                 (int32_t)parts, a.cols, dweight, dt);
  note_launches(1);
  return launch_status();
}

bool float_type(mp_dtype t) { return t == MP_F32 || t == MP_F16 || t == MP_BF16; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace
}  // namespace mp

extern "C" MP_API mp_status rmsnorm_residual_fp8(const void* x, const void* residual, mp_dtype x_dtype, int64_t rows,
                                                 int64_t cols, const void* weight, mp_dtype w_dtype, float eps,
                                                 void* h, void* y, mp_dtype fp8_dtype, int32_t scale_block,
                                                 void* y_scales, float* rstd, void* ckpt, float* ckpt_scales,
                                                 void* stream) {
  using namespace mp;
  if (rows < 0 || cols < 0) return MP_EINVAL;
  if (!float_type(x_dtype) || !float_type(w_dtype)) return MP_EINVAL;
  if (fp8_dtype != MP_E4M3 && fp8_dtype != MP_E5M2) return MP_EINVAL;
  if (scale_block != 128 && scale_block != 32) return MP_EINVAL;
  if (!(eps >= 0.0f && eps < INFINITY)) return MP_EINVAL;
  if (rows >= (1ll << 31) || cols > kMaxCols || cols % (scale_block == 32 ? 32 : 16) != 0) return MP_ESHAPE;
  if (rows == 0 || cols == 0) return MP_OK;
  if (!x || !weight || !y || !y_scales || (!ckpt != !ckpt_scales)) return MP_EINVAL;
  if (!aligned16(x) || !aligned16(residual) || !aligned16(weight) || !aligned16(h) || !aligned16(y) ||
      !aligned16(ckpt) || !aligned4(ckpt_scales) || !aligned4(rstd) || (scale_block == 128 && !aligned4(y_scales)))
    return MP_EALIGN;
  const int32_t tiles = (int32_t)((cols + kTile - 1) / kTile);
  NormFwd a;
  a.x = x, a.residual = residual, a.weight = weight, a.h = h, a.rstd = rstd;
  a.y = Fp8Out{static_cast<uint8_t*>(y), y_scales, scale_block == 32 ? (int32_t)(cols / 32) : tiles,
               fp8_dtype == MP_E5M2, scale_block == 32};
  a.ckpt = Fp8Out{static_cast<uint8_t*>(ckpt), ckpt_scales, tiles, false, false};
  a.rows = rows, a.cols = (int32_t)cols, a.wt = w_dtype, a.eps = eps;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (x_dtype) {
    case MP_F32: return launch_fwd_shape<XF32>(a, st);
    case MP_F16: return launch_fwd_shape<XF16>(a, st);
    default: return launch_fwd_shape<XBF16>(a, st);
  }
}

extern "C" MP_API size_t rmsnorm_workspace_size(int64_t rows, int64_t cols) {
  using namespace mp;
  if (rows <= 0 || cols <= 0 || cols > kMaxCols) return 0;
  return (size_t)parts_of(rows, cols) * (size_t)cols * sizeof(float);
}

extern "C" MP_API mp_status rmsnorm_residual_backward(const void* dy, const void* dh, mp_dtype x_dtype, int64_t rows,
                                                      int64_t cols, const void* h, const void* ckpt,
                                                      const float* ckpt_scales, const void* weight, mp_dtype w_dtype,
                                                      const float* rstd, void* dx, void* dweight, mp_dtype dw_dtype,
                                                      void* d_workspace, size_t workspace_bytes, void* stream) {
  using namespace mp;
  if (rows < 0 || cols < 0) return MP_EINVAL;
  if (!float_type(x_dtype) || !float_type(w_dtype) || !float_type(dw_dtype)) return MP_EINVAL;
  if (rows >= (1ll << 31) || cols > kMaxCols || cols % 16 != 0) return MP_ESHAPE;
  if (cols == 0) return MP_OK;
  if (!dweight) return MP_EINVAL;
  if (!aligned16(dweight)) return MP_EALIGN;
  if (rows > 0) {
    if (!dy || !weight || !rstd || !dx || (!ckpt != !ckpt_scales) || (!h == !ckpt)) return MP_EINVAL;
    if (!aligned16(dy) || !aligned16(dh) || !aligned16(h) || !aligned16(ckpt) || !aligned4(ckpt_scales) ||
        !aligned16(weight) || !aligned4(rstd) || !aligned16(dx))
      return MP_EALIGN;
    if (!d_workspace || workspace_bytes < rmsnorm_workspace_size(rows, cols)) return MP_EWORKSPACE;
    if (!aligned16(d_workspace)) return MP_EALIGN;
  }
  NormBwd a;
  a.dy = dy, a.dh = dh, a.h = h, a.weight = weight, a.codes = static_cast<const uint8_t*>(ckpt);
  a.scales = ckpt_scales, a.rstd = rstd, a.dx = dx, a.parts = static_cast<float*>(d_workspace);
  a.rows = rows, a.cols = (int32_t)cols, a.tiles = (int32_t)((cols + kTile - 1) / kTile), a.wt = w_dtype;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (x_dtype) {
    case MP_F32: return ckpt ? launch_bwd<XF32, true>(a, dweight, dw_dtype, st) : launch_bwd<XF32, false>(a, dweight, dw_dtype, st);
    case MP_F16: return ckpt ? launch_bwd<XF16, true>(a, dweight, dw_dtype, st) : launch_bwd<XF16, false>(a, dweight, dw_dtype, st);
    default: return ckpt ? launch_bwd<XBF16, true>(a, dweight, dw_dtype, st) : launch_bwd<XBF16, false>(a, dweight, dw_dtype, st);
  }
}
