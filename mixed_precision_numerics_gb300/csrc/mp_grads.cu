// mp_grads.cu — the global norm of a list of gradients, and their clipping.
//
//   norm = sqrt(sum over all tensors of g^2) / S,  c = min(1, max / (norm + 1e-6)),
//   out = g * c, in place or into tensors of another type: a binary32 product,
//   then rounded to that type.
//
// The optimizer's check pass (mp_adamw.cu) has the norm of one call's 16-bit
// gradients, for that call alone.  These two calls are for what it does not
// cover: several parameter groups under one norm, and gradients accumulated in
// FP32 that are clipped into the 16-bit ones which the step reads.
//
// Squares are summed in binary32 over the 64 elements that a thread holds (32
// in FP32), where they neither overflow nor vanish; elsewhere the thread's
// elements are scaled by the power of two of their largest first.  Those sums
// are added in binary64, in an order fixed by the list and the device.
//
// Bound by DRAM: the norm reads every gradient once; the clipping reads and
// writes it.  The clipping walks the list backwards, so that it begins with
// what the norm has left in L2.  839M BF16 gradients: norm 236 us (7.1 TB/s),
// clipping 525 (6.4), both 761, which is 0.98 of three passes at the copy rate;
// 81M FP32 into FP16 118 us, 1.0.  Three CTAs an SM, 96 KB of loads in flight:
// four have 64 registers a thread and spill (norm 300 us).  Few small tensors are
// the latency of two launches (20 tensors of 2.6M elements 9.8 us on the GPU).
#include <new>

#include "mp_chain.cuh"
#include "mp_device.cuh"
#include "mp_internal.h"
#include "mp_tile8.cuh"

namespace mp {
namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 8;                             // 16-byte loads in flight a thread
constexpr int kTileElems = kThreads * kVecs * 8;     // of a CTA's step
constexpr int kCap = 512, kFew = 32;                 // tensors a launch
constexpr int kNormCtas = 3, kClipCtas = 3;          // an SM

struct Grad {
  const void* g;
  void* out;
  int64_t n;
  int32_t gt, ot;  // mp_dtype
};
template <int CAP>
struct List {
  int64_t start[CAP + 1];  // prefix sums of the tensors' tiles
  Grad t[CAP];
  int32_t count;
};

// The tensor of a tile, from that of an earlier one (every listed tensor has a tile).
template <int CAP>
__device__ __forceinline__ int tensor_of(const List<CAP>& L, int64_t tile, int i) {
  if (tile < L.start[i + 1]) return i;
  int lo = i + 1, hi = L.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (L.start[mid] <= tile) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

template <int XT>
constexpr int kVecElems = XT == XF32 ? 4 : 8;

// A thread's vectors of one of a tile's kGroups<XT> parts, from element `at`.
template <int XT>
constexpr int kGroups = kTileElems / (kThreads * kVecs * kVecElems<XT>);
template <int XT>
__device__ __forceinline__ void load_vecs(uint4 (&v)[kVecs], const void* g, int64_t at, int64_t n, bool whole) {
  constexpr int V = kVecElems<XT>;
  const uint4* p = reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(g) + at * (16 / V));
  if (whole) {
#pragma unroll
    for (int u = 0; u < kVecs; ++u) v[u] = p[u * kThreads];
  } else {  // the tensor's last tile: zeros from its last whole vector on
#pragma unroll
    for (int u = 0; u < kVecs; ++u) v[u] = at + u * kThreads * V + V <= n ? p[u * kThreads] : make_uint4(0u, 0u, 0u, 0u);
  }
}
// The elements behind a tensor's last whole vector are a thread's each: its number, or -1.
template <int XT>
__device__ __forceinline__ int64_t end_of(int64_t n, bool whole) {
  const int rest = (int)(n & (kVecElems<XT> - 1));
  return !whole && threadIdx.x < rest ? n - rest + threadIdx.x : -1;
}
template <int XT>
__device__ __forceinline__ float element(const void* g, int64_t e) {
  if constexpr (XT == XF32) return static_cast<const float*>(g)[e];
  const uint32_t w = static_cast<const uint16_t*>(g)[e];
  return XT == XF16 ? f16lo(w) : bf16lo(w);
}

// Element pairs of 16 bytes.
template <int XT>
__device__ __forceinline__ float2 vec_pair(uint4 q, int k) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  if constexpr (XT == XF32)
    return make_float2(__uint_as_float(w[2 * k]), __uint_as_float(w[2 * k + 1]));
  else if constexpr (XT == XF16)
    return make_float2(f16lo(w[k]), f16hi(w[k]));
  else
    return make_float2(bf16lo(w[k]), bf16hi(w[k]));
}

// Sum of squares of a thread's vectors, in binary64.
template <int XT>
__device__ __forceinline__ double squares(const uint4 (&v)[kVecs]) {
  float2 a = both(0.0f), b = both(0.0f);
#pragma unroll
  for (int u = 0; u < kVecs; ++u)
#pragma unroll
    for (int k = 0; k < kVecElems<XT> / 2; k += 2) {
      const float2 x = vec_pair<XT>(v[u], k), y = vec_pair<XT>(v[u], k + 1);
      a = fma2(x, x, a);
      b = fma2(y, y, b);
    }
  a = add2(a, b);
  const float s = a.x + a.y;
  // FP16's squares are between 2^-48 and 2^33.
  if (XT == XF16 || (s > 0x1p-80f && s < 0x1p+100f)) return (double)s;
  float m = 0.0f;
#pragma unroll
  for (int u = 0; u < kVecs; ++u)
#pragma unroll
    for (int k = 0; k < kVecElems<XT> / 2; ++k) {
      const float2 x = vec_pair<XT>(v[u], k);
      m = max3_abs_nan(m, x.x, x.y);
    }
  if (m == 0.0f || !(m < INFINITY)) return (double)s;  // 0, infinity or NaN
  const int e = max((int)(__float_as_uint(m) >> 23), 1);
  const float2 down = both(e < 254 ? __uint_as_float((uint32_t)(254 - e) << 23) : 0x1p-127f);  // 2^(127 - e)
  float2 c = both(0.0f);
#pragma unroll
  for (int u = 0; u < kVecs; ++u)
#pragma unroll
    for (int k = 0; k < kVecElems<XT> / 2; ++k) {
      const float2 x = mul2(vec_pair<XT>(v[u], k), down);
      c = fma2(x, x, c);
    }
  return (double)(c.x + c.y) * __longlong_as_double((long long)(1023 + 2 * (e - 127)) << 52);
}

template <int XT>
__device__ __forceinline__ double tile_squares(const Grad& t, int64_t base) {
  constexpr int V = kVecElems<XT>;
  const bool whole = base + kTileElems <= t.n;
  double s = 0.0;
#pragma unroll
  for (int h = 0; h < kGroups<XT>; ++h) {
    uint4 v[kVecs];
    const int64_t at = base + (int64_t)h * kThreads * kVecs * V + threadIdx.x * V;
    load_vecs<XT>(v, t.g, at, t.n, whole);
    s += squares<XT>(v);
  }
  if (const int64_t e = end_of<XT>(t.n, whole); e >= 0) {
    const double x = element<XT>(t.g, e);
    s += x * x;
  }
  return s;
}

template <int LANES>
__device__ __forceinline__ double lane_sum(double v) {
#pragma unroll
  for (int h = LANES / 2; h >= 1; h >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, h);
  return v;
}
// In thread 0.
__device__ __forceinline__ double block_sum(double v, double* ws) {
  v = lane_sum<32>(v);
  if ((threadIdx.x & 31) == 0) ws[threadIdx.x >> 5] = v;
  __syncthreads();
  return threadIdx.x < 32 ? lane_sum<kThreads / 32>(ws[threadIdx.x & (kThreads / 32 - 1)]) : 0.0;
}

// Each CTA's sum goes to sums[first + its number]; with `last` the CTA that
// finishes last (an atomic ticket, no waiting) adds all `first + gridDim.x` of
// them in order and leaves the ticket at zero.
template <int CAP>
__global__ __launch_bounds__(kThreads, kNormCtas) void k_grad_norm(const __grid_constant__ List<CAP> L, double* sums,
                                                                   int32_t first, uint32_t* ticket, bool last,
                                                                   const float* loss_scale, float* norm) {
  __shared__ double ws[kThreads / 32];
  __shared__ bool fold;
  chain_wait();
  chain_release();
  const int64_t total = L.start[L.count];
  double s = 0.0;
  int i = 0;
  for (int64_t tile = blockIdx.x; tile < total; tile += gridDim.x) {
    i = tensor_of(L, tile, i);
    const Grad& t = L.t[i];
    const int64_t base = (tile - L.start[i]) * kTileElems;
    s += t.gt == XF32 ? tile_squares<XF32>(t, base)
                      : t.gt == XF16 ? tile_squares<XF16>(t, base) : tile_squares<XBF16>(t, base);
  }
  s = block_sum(s, ws);
  if (threadIdx.x == 0) {
    sums[first + blockIdx.x] = s;
    fold = false;
    if (last) {
      __threadfence();
      fold = atomicAdd(ticket, 1u) == gridDim.x - 1;
    }
  }
  __syncthreads();
  if (!fold) return;
  __threadfence();
  s = 0.0;
  for (int i = threadIdx.x; i < first + (int)gridDim.x; i += kThreads) s += __ldcg(sums + i);
  s = block_sum(s, ws);
  if (threadIdx.x == 0) {
    s = sqrt(s);
    *norm = (float)(loss_scale ? s / (double)*loss_scale : s);
    *ticket = 0u;
  }
}

template <int XT, int OT>
__device__ __forceinline__ void clip_tile(const Grad& t, int64_t base, float c) {
  constexpr int V = kVecElems<XT>;
  const bool whole = base + kTileElems <= t.n;
#pragma unroll
  for (int h = 0; h < kGroups<XT>; ++h) {
    uint4 v[kVecs];
    const int64_t at = base + (int64_t)h * kThreads * kVecs * V + threadIdx.x * V;
    load_vecs<XT>(v, t.g, at, t.n, whole);
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      const int64_t e = at + u * kThreads * V;
      constexpr int W = V / (OT == XF32 ? 1 : 2);  // words out
      uint32_t w[W];
#pragma unroll
      for (int k = 0; k < V / 2; ++k) {
        const float2 x = mul2(vec_pair<XT>(v[u], k), both(c));
        if constexpr (OT == XF32) {
          w[2 * k] = __float_as_uint(x.x), w[2 * k + 1] = __float_as_uint(x.y);
        } else if constexpr (OT == XF16) {
          asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[k]) : "f"(x.y), "f"(x.x));
        } else {
          asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[k]) : "f"(x.y), "f"(x.x));
        }
      }
      if (whole || e + V <= t.n) {
        uint32_t* to = static_cast<uint32_t*>(t.out) + e * W / V;
        if constexpr (W == 2) {
          __stcs(reinterpret_cast<uint2*>(to), make_uint2(w[0], w[1]));
        } else {
#pragma unroll
          for (int i = 0; i < W; i += 4) st_cs(to + i, make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]));
        }
      }
    }
  }
  if (const int64_t e = end_of<XT>(t.n, whole); e >= 0) {
    const float x = element<XT>(t.g, e) * c;
    if constexpr (OT == XF32)
      static_cast<float*>(t.out)[e] = x;
    else
      static_cast<uint16_t*>(t.out)[e] = (uint16_t)(OT == XF16 ? pack_f16x2(x, 0.0f) : pack_bf16x2(x, 0.0f));
  }
}
template <int XT>
__device__ __forceinline__ void clip_tile(const Grad& t, int64_t base, float c) {
  if (t.ot == XF32) clip_tile<XT, XF32>(t, base, c);
  else if (t.ot == XF16) clip_tile<XT, XF16>(t, base, c);
  else clip_tile<XT, XBF16>(t, base, c);
}

template <int CAP>
__global__ __launch_bounds__(kThreads, kClipCtas) void k_grad_clip(const __grid_constant__ List<CAP> L,
                                                                   const float* norm, float max_norm) {
  __shared__ float factor;
  chain_wait();
  chain_release();
  if (threadIdx.x == 0) {
    const float n = __ldcg(norm);
    const double c = __ddiv_rn((double)max_norm, __dadd_rn((double)n, 1e-6));
    factor = n < INFINITY ? (float)fmin(c, 1.0) : __uint_as_float(0x7FFFFFFFu);
  }
  __syncthreads();
  const float c = factor;
  const int64_t total = L.start[L.count];
  int i = 0;
  for (int64_t tile = blockIdx.x; tile < total; tile += gridDim.x) {
    i = tensor_of(L, tile, i);
    const Grad& t = L.t[i];
    if (c == 1.0f && t.g == t.out) continue;  // nothing changes
    const int64_t base = (L.start[i + 1] - 1 - tile) * kTileElems;  // from the tensor's end
    if (t.gt == XF32) clip_tile<XF32>(t, base, c);
    else if (t.gt == XF16) clip_tile<XF16>(t, base, c);
    else clip_tile<XBF16>(t, base, c);
  }
}

bool float_type(mp_dtype t) { return t == MP_F32 || t == MP_F16 || t == MP_BF16; }

// Tensors that have elements: how many, in how many tiles.
struct Extent {
  int64_t count = 0, tiles = 0;
};
Extent extent_of(const mp_grad* g, int32_t n) {
  Extent x;
  for (int32_t i = 0; i < n; ++i)
    if (g[i].numel > 0) ++x.count, x.tiles += (g[i].numel + kTileElems - 1) / kTileElems;
  return x;
}
int64_t launches_of(const Extent& x) { return x.count <= kFew ? 1 : (x.count + kCap - 1) / kCap; }
int most_ctas() { return sm_count() * kNormCtas; }

// An empty gradient has types and nothing else: its pointers are not looked at.
mp_status check(const mp_grad* g, int32_t n, bool outs) {
  if (n < 0 || (n > 0 && !g)) return MP_EINVAL;
  for (int32_t i = 0; i < n; ++i) {
    if (g[i].numel < 0 || !float_type(g[i].grad_dtype) || (outs && !float_type(g[i].out_dtype))) return MP_EINVAL;
    if (g[i].numel == 0) continue;
    if (!g[i].grad || (outs && !g[i].out)) return MP_EINVAL;
    if (outs && g[i].out == g[i].grad && g[i].out_dtype != g[i].grad_dtype) return MP_EINVAL;
  }
  for (int32_t i = 0; i < n; ++i)
    if (g[i].numel > 0 && (!aligned16(g[i].grad) || (outs && !aligned16(g[i].out)))) return MP_EALIGN;
  return MP_OK;
}

// Calls launch(list) for lists of up to CAP tensors, in the caller's order or from its end.
template <int CAP, typename Launch>
mp_status in_lists(const mp_grad* g, int32_t n, bool backwards, Launch launch) {
  List<CAP>* L = new (std::nothrow) List<CAP>;
  if (!L) return MP_ECUDA;
  mp_status st = MP_OK;
  L->count = 0, L->start[0] = 0;
  for (int32_t j = 0; j < n && st == MP_OK; ++j) {
    const mp_grad& t = g[backwards ? n - 1 - j : j];
    if (t.numel > 0) {
      L->t[L->count] = Grad{t.grad, t.out, t.numel, t.grad_dtype, t.out_dtype};
      L->start[L->count + 1] = L->start[L->count] + (t.numel + kTileElems - 1) / kTileElems;
      ++L->count;
    }
    if (L->count == CAP) {
      st = launch(*L);
      L->count = 0;
    }
  }
  if (L->count && st == MP_OK) st = launch(*L);
  delete L;
  return st;
}

template <int CAP>
mp_status norm_of(const mp_grad* g, int32_t n, const Extent& x, const float* loss_scale, float* norm, void* ws,
                  cudaStream_t st) {
  uint32_t* ticket = static_cast<uint32_t*>(ws);
  double* sums = reinterpret_cast<double*>(static_cast<unsigned char*>(ws) + 64);
  int64_t left = x.count;
  int32_t first = 0;
  return in_lists<CAP>(g, n, false, [&](const List<CAP>& L) {
    left -= L.count;
    const int grid = grid_for(L.start[L.count], kNormCtas);
    launch_chained(k_grad_norm<CAP>, dim3(grid), dim3(kThreads), 0, st, L, sums, first, ticket, left == 0, loss_scale,
                   norm);
    first += grid;
    note_launches(1);
    return launch_status();
  });
}

template <int CAP>
mp_status clip_all(const mp_grad* g, int32_t n, const float* norm, float max_norm, cudaStream_t st) {
  return in_lists<CAP>(g, n, true, [&](const List<CAP>& L) {
    launch_chained(k_grad_clip<CAP>, dim3(grid_for(L.start[L.count], kClipCtas)), dim3(kThreads), 0, st, L, norm, max_norm);
    note_launches(1);
    return launch_status();
  });
}

}  // namespace
}  // namespace mp

extern "C" MP_API size_t mp_grad_norm_workspace_size(const mp_grad* grads, int32_t n) {
  using namespace mp;
  if (n < 0 || (n > 0 && !grads)) return 0;
  return 64 + (size_t)launches_of(extent_of(grads, n)) * most_ctas() * sizeof(double);
}

extern "C" MP_API mp_status mp_grad_norm(const mp_grad* grads, int32_t n, const float* d_loss_scale, float* d_norm,
                                         void* d_workspace, size_t workspace_bytes, void* stream) {
  using namespace mp;
  if (const mp_status s = check(grads, n, false); s != MP_OK) return s;
  if (!d_norm) return MP_EINVAL;
  if ((reinterpret_cast<uintptr_t>(d_norm) & 3u) || (reinterpret_cast<uintptr_t>(d_loss_scale) & 3u) ||
      !aligned16(d_workspace))
    return MP_EALIGN;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const Extent x = extent_of(grads, n);
  if (x.count == 0) return cudaMemsetAsync(d_norm, 0, 4, st) == cudaSuccess ? MP_OK : MP_ECUDA;
  if (!d_workspace || workspace_bytes < mp_grad_norm_workspace_size(grads, n)) return MP_EWORKSPACE;
  return x.count <= kFew ? norm_of<kFew>(grads, n, x, d_loss_scale, d_norm, d_workspace, st)
                         : norm_of<kCap>(grads, n, x, d_loss_scale, d_norm, d_workspace, st);
}

extern "C" MP_API mp_status mp_grad_clip(const mp_grad* grads, int32_t n, const float* d_norm, float max_norm,
                                         void* stream) {
  using namespace mp;
  if (const mp_status s = check(grads, n, true); s != MP_OK) return s;
  if (!d_norm || !(max_norm > 0.0f) || !(max_norm < INFINITY)) return MP_EINVAL;
  if (reinterpret_cast<uintptr_t>(d_norm) & 3u) return MP_EALIGN;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return extent_of(grads, n).count <= kFew ? clip_all<kFew>(grads, n, d_norm, max_norm, st)
                                           : clip_all<kCap>(grads, n, d_norm, max_norm, st);
}
