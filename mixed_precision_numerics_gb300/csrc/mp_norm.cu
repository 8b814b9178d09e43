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
// Both read and write every element once, and are bound by DRAM: a row stays on
// its SM between the two uses of it, before and after the row's sum.  Forward
// it stays in registers; backward, where the column sums dw take those, in
// shared memory.  [8192 x 4096] BF16 with checkpoint: forward 42.6 us, 0.94 of
// the copy rate (6793 GB/s), backward 42.1 us, 0.82; [16384 x 5120]: 101.4 us,
// 0.98, and 94.8 us, 0.92.
#include <math.h>

#include "mp_chain.cuh"
#include "mp_internal.h"
#include "mp_tile8.cuh"

namespace mp {
namespace {

constexpr int kCta = 256;           // threads of a CTA that takes several rows at a time
constexpr int kMaxThreads = 1024;   // threads of a CTA that takes one row at a time
constexpr int kMaxCols = kMaxThreads * kUnit;
constexpr int64_t kMaxRows = (1ll << 31) - 32;  // a row's number and that of its group's last are 32-bit
constexpr int kMaxParts = 608;      // partial sums of dweight: four CTAs on each of 152 SMs

// How a row is laid over threads, by its length alone: `lanes` of a warp (8,
// 16 or 32) and kCta / lanes rows a CTA, or (lanes 0) a CTA of `threads`, one
// 16-element unit a thread.  Instead of either, a row may lie in whole tiles (of
// eight lanes) of a CTA or team: in_tiles, tiles_save_lanes.
struct RowShape {
  int lanes, threads, rows_per_cta;
};
RowShape row_shape(int64_t cols) {
  const int n = (int)(cols / kUnit);
  if (n > 32) return {0, (n + 31) / 32 * 32, 1};
  const int l = n <= 8 ? 8 : n <= 16 ? 16 : 32;
  return {l, kCta, kCta / l};
}
constexpr int kSmemBytes = 224 * 1024;   // dynamic shared memory of a CTA that has an SM to itself
constexpr int kSmemShared = 216 * 1024;  // of all CTAs that share one

// Threads that hold such a row with `u` units each.
int team_of(const RowShape& s, int u) { return (s.threads / u + 31) / 32 * 32; }
// CTAs that take `groups` groups of rows in turn, `per_sm` resident on an SM.
int resident_grid(int64_t groups, int per_sm) {
  const int64_t most = (int64_t)sm_count() * (per_sm < 1 ? 1 : per_sm);
  return (int)(groups < most ? groups : most);
}

// Raises a kernel's dynamic shared-memory limit where a launch may need more
// than the default: 48 KB, the kernel's static arrays included.
template <typename K>
bool smem_ok(K kernel, int bytes, std::atomic<uint64_t>& done) {
  return bytes <= 32 * 1024 || smem_opt_in(kernel, kSmemBytes, done);
}

// Brings bytes (a multiple of 16, as their address is) into L2.
__device__ __forceinline__ void prefetch_l2(const void* at, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(__cvta_generic_to_global(at)), "r"(bytes) : "memory");
}

// Sum over the L lanes that hold one row, in every one of them.
template <int L>
__device__ __forceinline__ float lane_sum(float v) {
#pragma unroll
  for (int d = L / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  return v;
}
// Sum over the row's tiles of eight lanes each, at most kTilesMax of them, in
// every lane of the row; slot: a float for each.  All of the CTA's threads call.
__device__ __forceinline__ float tiles_sum(float v, float* slot, int tiles, int u) {
  v = lane_sum<8>(v);
  const int i = u & 7;
  if (i == 0) slot[u >> 3] = v;
  __syncthreads();
  return lane_sum<8>((i < tiles ? slot[i] : 0.0f) + (i + 8 < tiles ? slot[i + 8] : 0.0f));
}
// Sum over the CTA's threads and their U units, in every one of them.  Units 32 b
// to 32 b + 31 are added up first, whatever U is, so that a row's sum does not
// depend on how many rows the call has; slots: 32 floats.
template <int U>
__device__ __forceinline__ float cta_sum(float (&v)[U], float* slots) {
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
#pragma unroll
  for (int k = 0; k < U; ++k) {
    v[k] = lane_sum<32>(v[k]);
    if (lane == 0) slots[(threadIdx.x >> 5) + k * warps] = v[k];
  }
  __syncthreads();
  return lane_sum<32>(lane < U * warps ? slots[lane] : 0.0f);
}
// The same of N sums, in a team of `threads`; slot: N floats for each tile of the
// team.  It must not be written again before every thread has passed the next
// barrier: callers alternate between two.
template <int N>
__device__ __forceinline__ void tiles_sums(float (&v)[N], float* slot, int barrier, int t, int threads, int tiles,
                                           int sub) {
  const int i = t & 7;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    v[k] = lane_sum<8>(v[k]);
    if (i == 0) slot[(t >> 3) * N + k] = v[k];
  }
  named_barrier(barrier, threads);
  const float* row = slot + sub * tiles * N;
#pragma unroll
  for (int k = 0; k < N; ++k)
    v[k] = lane_sum<8>((i < tiles ? row[i * N + k] : 0.0f) + (i + 8 < tiles ? row[(i + 8) * N + k] : 0.0f));
}
// N sums over the `threads` of a team (whole warps; t the thread's place in it),
// in a fixed order, in every one of them.  `slot` (N floats for each warp) must
// not be written again before every thread has passed the next barrier:
// callers alternate between two.
template <int N>
__device__ __forceinline__ void team_sums(float (&v)[N], float* slot, int barrier, int t, int threads) {
  const int lane = t & 31;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    v[k] = lane_sum<32>(v[k]);
    if (lane == 0) slot[(t >> 5) * N + k] = v[k];
  }
  named_barrier(barrier, threads);
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = lane_sum<32>(lane < (threads >> 5) ? slot[lane * N + k] : 0.0f);
}

// ---------------------------------------------------------------------------
// Forward
// ---------------------------------------------------------------------------
constexpr int kInTiles = 1;    // a layout beside 8, 16 and 32 lanes: see in_tiles
constexpr int kTilesMax = 16;  // tiles of its rows
struct NormFwd {
  const void *x, *residual, *weight;
  void* h;
  float* rstd;
  Fp8Out y;
  uint8_t* ckpt;
  float* ckpt_scales;
  int64_t rows;
  int32_t cols, tiles, wt;
  int32_t group;  // rows of a CTA, where L is kInTiles
  float eps, inv_cols;
};

// A row lies in L lanes of a warp, in tiles of eight lanes of a CTA that holds
// `group` rows (L = kInTiles) or in the whole CTA (L = 0), U units a thread:
// unit k of thread t is t + k * threads.  Every CTA is launched at once; the
// others on the SM keep DRAM busy while one meets its row's barrier.
// Dropped: CTAs that stay and fetch the next rows into shared memory a thread
// at a time, 60.2 us on [8192 x 4096] BF16 against 42.8; a cluster of CTAs for a
// row, 130 us on [16384 x 5120]; the rows of the next wave sent for as far as L2
// (43.5 us on [8192 x 4096] against 42.6, 100.7 on [16384 x 5120] against 101.3).
template <int XT, int L, int U>
constexpr int fwd_threads() { return L == kInTiles ? 512 : L ? kCta : U == 1 ? kMaxThreads : XT == XF32 ? 768 : kMaxThreads / 2; }
template <int XT, int L, int U, bool SAVE>
__global__ __launch_bounds__(fwd_threads<XT, L, U>(), XT != XF32 && U == 2 ? 2 : 1) void k_norm_fwd(const __grid_constant__ NormFwd a) {
  __shared__ float slots[L == kInTiles ? 5 * kTilesMax : 32];
  chain_wait();
  chain_release();
  const int units = a.cols / kUnit, T = blockDim.x;
  int u = threadIdx.x, sub = 0, R = 1;  // the thread's unit, its row among the CTA's, their number
  if constexpr (L == kInTiles) {
    sub = u / (a.tiles * 8);
    u -= sub * a.tiles * 8;
    R = a.group;
  } else if constexpr (L > 0) {
    sub = u / L;
    u %= L;
    R = kCta / L;
  }
  // Threads past the last of `group` rows, less than a row of them, have none.
  const int64_t row = L == kInTiles && sub >= R ? a.rows : (int64_t)blockIdx.x * R + sub;
  Place p[U];
  Unit<XT> h[U][2], r[U];
  Weights w;
#pragma unroll
  for (int k = 0; k < U; ++k) {
    p[k].row = (int32_t)row;
    p[k].u = u + k * T;
    p[k].at = row * a.cols + p[k].u * kUnit;
    p[k].in = row < a.rows && p[k].u < units;
    p[k].tile_in = row < a.rows && (p[k].u & ~7) < units;
    h[k][0].zero();
    r[k].zero();
    if (p[k].in) {
      h[k][0].load(a.x, p[k].at);
      if (a.residual) r[k].load(a.residual, p[k].at);
      if constexpr (U == 1) w.load(a.weight, a.wt, p[k].u);
    }
  }
  float part[U], amax[U];
#pragma unroll
  for (int k = 0; k < U; ++k) {
    if (a.residual) h[k][0].add(r[k]);
    if (p[k].in && a.h) h[k][0].store(a.h, p[k].at);
    float2 ss = both(0.0f);
    amax[k] = 0.0f;
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const float2 f = h[k][0].pair(i);
      ss = fma2(f, f, ss);
      if constexpr (SAVE) amax[k] = max3_abs_nan(amax[k], f.x, f.y);
    }
    part[k] = ss.x + ss.y;
  }
  const float sum = L == kInTiles ? tiles_sum(part[0], slots + sub * kTilesMax, a.tiles, u)
                    : L           ? lane_sum<L ? L : 1>(part[0])
                                  : cta_sum(part, slots);
  // In binary32: within 3 * 2^-24 of 1 / sqrt(mean + eps) on random rows, as a correctly rounded division and root
  // of the same sum are (the sum's own error is the larger part).
  const float rstd = rsqrtf(fmaf(sum, a.inv_cols, a.eps));
  if (u == 0 && row < a.rows && a.rstd) a.rstd[row] = rstd;
#pragma unroll
  for (int k = 0; k < U; ++k) {
    if (k > 0 && !__any_sync(0xFFFFFFFFu, p[k].in)) break;  // no lane of the warp has a second unit
    float2 y[kPairs];
    if constexpr (U > 1) w.load(a.weight, a.wt, min(p[k].u, units - 1));
    w.floats(a.wt, y);
    h[k][0].forget();
#pragma unroll
    for (int i = 0; i < kPairs; ++i) y[i] = mul2(mul2(h[k][0].pair(i), both(rstd)), y[i]);
    if constexpr (SAVE) {
      const uint32_t mc[2] = {tile_max(__float_as_uint(amax[k])), 0u};
      uint8_t* const cc[2] = {a.ckpt, nullptr};
      float* const cs[2] = {a.ckpt_scales, nullptr};
      cast_store<2, XT>(y, a.y, p[k], mc, h[k], cc, cs, a.tiles);
    } else {
      cast_store<XT>(y, a.y, p[k]);
    }
  }
}

template <int XT, int L, int U, bool SAVE>
mp_status launch_fwd(const NormFwd& a, const RowShape& s, cudaStream_t st) {
  const int rows = L == kInTiles ? a.group : s.rows_per_cta;
  const int threads = L == kInTiles ? (rows * a.tiles + 3) / 4 * 32 : L ? kCta : team_of(s, U);
  const int64_t groups = (a.rows + rows - 1) / rows;  // below 2^31
  launch_chained(k_norm_fwd<XT, L, U, SAVE>, dim3((unsigned)groups), dim3(threads), 0, st, a);
  note_launches(1);
  return launch_status();
}

// Rows that do not fill their warps, in tiles instead.  BF16 with the checkpoint,
// GPU time in us over inputs beyond L2 with this layout and with whole warps: [16384
// x 576] 15.3 and 19.0, [1024 x 768] 3.1 and 3.3, [16384 x 1040] 27.1 and 30.1,
// [16384 x 1280] 28.3 and 31.8, [16384 x 384] 10.2 and 11.7, [16384 x 1536] 32.2 and
// 33.4, [16384 x 2048] 41.3 and 42.3, but 40.4 and 38.2 at 1792.  Four tiles are a
// warp, whose rows need no barrier: [16384 x 512] 9.8, and 17.3 in this layout.
// FP32 is nearer to DRAM: [16384 x 576] 23.4 and 25.2, but [4096 x 896] 11.1 and
// 10.3, [16384 x 384] 16.6 and 15.8.
template <int XT>
bool in_tiles(int tiles) {
  return XT == XF32 ? tiles == 5 || tiles == 6 : tiles >= 3 && tiles <= kTilesMax && tiles != 4;
}
// Rows of a CTA in that layout: as many as let the most tiles be on an SM.
int rows_in_tiles(int tiles) {
  int best = 1, most = 0;
  for (int rows = 1; rows <= 4; ++rows) {  // with four no lane is idle
    const int warps = (rows * tiles + 3) / 4, held = kMaxThreads / 32 / warps * rows;
    if (held > most) most = held, best = rows;
  }
  return best;
}
// Whether a CTA that takes one row holds one unit a thread, and not two.  One
// has its weights by the row's sum, where two (in the 16-bit types) read them
// after it, to be 64 registers (with 8 bytes a thread spilled, and with the
// checkpoint 28) and to have twice the rows on an SM.  That counts
// once the rows come in several waves, the earlier the fewer fit on an SM.  BF16,
// us with one and with two: one row of 4096 2.1 and 2.8, [37 x 5120] 2.1 and 2.9,
// [1024 x 4096] 7.8 and 8.3, [304 x 16384] 10.2 and 9.1, [8192 x 4096] 42.5 and
// 42.4, [16384 x 5120] 107.2 and 101.1.  FP32 has 80 registers with two, and is
// better off with one up to 8192 columns ([7000 x 4096] 64.3 and 71.5; [7000 x
// 10816] 223.7 and 188.4).
template <int XT>
bool one_unit(const RowShape& s, int64_t rows) {
  const int held = kMaxThreads / s.threads;
  return (XT == XF32 && held > 1) || rows <= (int64_t)sm_count() * held * (held < 3 ? held : 3);
}

template <int XT, bool SAVE>
mp_status launch_fwd_shape(NormFwd a, cudaStream_t st) {
  const RowShape s = row_shape(a.cols);
  if (in_tiles<XT>(a.tiles)) {
    a.group = rows_in_tiles(a.tiles);
    return launch_fwd<XT, kInTiles, 1, SAVE>(a, s, st);
  }
  if (s.lanes == 8) return launch_fwd<XT, 8, 1, SAVE>(a, s, st);
  if (s.lanes == 16) return launch_fwd<XT, 16, 1, SAVE>(a, s, st);
  if (s.lanes == 32) return launch_fwd<XT, 32, 1, SAVE>(a, s, st);
  return one_unit<XT>(s, a.rows) ? launch_fwd<XT, 0, 1, SAVE>(a, s, st) : launch_fwd<XT, 0, 2, SAVE>(a, s, st);
}
template <int XT>
mp_status launch_fwd_type(const NormFwd& a, cudaStream_t st) {
  return a.ckpt ? launch_fwd_shape<XT, true>(a, st) : launch_fwd_shape<XT, false>(a, st);
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
  int32_t team;     // threads of a team
  int32_t group;    // of its rows, one unit a thread, where L is kInTiles
  int32_t stages;   // of its ring
  bool stage_dh;    // whether dh comes through it
  float inv_cols;
};

constexpr int kMaxStages = 4;
constexpr int kMaxTeams = 15;            // a named barrier each
constexpr int kRowsThreads = 640;        // threads of 96 registers on an SM

__device__ unsigned int g_norm_wait_failures;  // bounded waits that gave up (read by mp_wait_failures)

// A group of rows comes through two rings of shared memory, by when its bytes
// are done with: `early` (dy) before the row's sum, `late` (the stream or its
// codes, read before and after the sum, then dh) after it.  Bytes of one stage
// of each, of a group of so many elements.
template <int XT>
__host__ __device__ constexpr int early_bytes(int elements) { return elements * (XT == XF32 ? 4 : 2); }
template <int XT, bool SAVED>
__host__ __device__ constexpr int late_bytes(int elements, bool dh) {
  return elements * ((SAVED ? 1 : XT == XF32 ? 4 : 2) + (dh ? (XT == XF32 ? 4 : 2) : 0));
}

// Bytes of the weights in binary32, the units a multiple of four so that each
// 16-byte piece of them starts on a multiple of 64 bytes.
__host__ __device__ constexpr int weight_bytes(int units) { return (units + 3) / 4 * 4 * kUnit * 4; }

// A CTA holds `teams` of threads (as many as the SM's registers take, where a
// row needs a whole team; one, where rows lie in a warp's lanes).  A team takes
// every (gridDim.x * teams)-th group of rows.  Its first thread keeps the
// team's rings filled with bulk copies (a group's rows are consecutive in
// memory, so a tensor's part of a group is one copy): an early stage is free
// after the barrier of the group's sum and is filled again there; a late one
// when the last of the team's warps has arrived at its `done` barrier, which
// the thread looks at when it begins the next group.  Each thread keeps the
// sums of its own columns in registers over its rows (binary32, in row order);
// at the end the CTA joins its teams' sums and writes one row of `parts`.
// Where a row needs a team, each thread has two slots: two units of a row or,
// with ROWS, one unit of two rows, which share the weights, the column sums and
// all that comes once a group.  With L = kInTiles a team has `group` rows beside
// each other, in tiles of eight lanes (and as many more in the second slots).
// Across the barrier of the sum live only the column sums and dy * w; the
// stream's values are converted twice.  A thread whose wait gave up works on what
// it finds and stores nothing more, but keeps meeting the barriers.
//
// [8192 x 4096] BF16 from the checkpoint, both kernels: with loads into
// registers 65.9 us, a ring of bulk copies 47.7, two units a thread (a row's
// waits, sum and addresses shared by twice the elements) 45.7, the weights in
// binary32 in shared memory, the late ring refilled early and no bank conflicts
// 43.4, two rows a team instead of two units 42.1 (38.1 within a
// graph).  Of the rest about 6 us are the first rows' latency, the last round, the
// join of the column sums and the second kernel (2.7).
//
// From the kept BF16 stream, within a graph: [8192 x 4096] 45.6 us, [16384 x 5120]
// 104.0 (floors 39.5 and 98.8).
//
// ONE: rows so long that there is room for one stage would meet all of DRAM's
// latency each time; so the next group's bytes are sent for as far as L2.  Those are
// FP32 rows from 8208 columns on from the stream and from 10432 on from the
// checkpoint, without dh from 11472 on from the stream, and 16-bit rows with dh from
// 14352 on from the stream.  FP32 [7000 x 12288] from the checkpoint 191 us, without
// the prefetch 225; [7000 x 9216] from the stream 164 and 201.
//
// Rows in lanes of a warp, from the checkpoint, spill 4 bytes a thread in the 16-bit
// types and 16 in FP32 at their 64 registers.
template <int XT, bool SAVED, int L, int U, bool ROWS, bool ONE>
__global__ __maxnreg__(U == 1 ? 64 : ROWS ? 96 : 128) void k_norm_bwd(const __grid_constant__ NormBwd a) {
  constexpr int NR = ROWS ? U : 1, NU = ROWS ? 1 : U;  // rows of a thread, and units in each
  extern __shared__ __align__(128) unsigned char smem[];
  constexpr bool kLanes = L > kInTiles, kTiles = L == kInTiles;
  constexpr int kSlots = kTiles ? kRowsThreads / 8 + kTilesMax : 32;  // a thread without a row reads up to a row past
  __shared__ float slots[2 * kSlots * NR];
  __shared__ uint64_t bars[kMaxTeams * 3 * kMaxStages];
  constexpr int es = XT == XF32 ? 4 : 2, ves = SAVED ? 1 : es;
  const int R1 = kTiles ? a.group : kLanes ? kCta / (L ? L : 1) : 1, R = R1 * NR;
  const int units = a.cols / kUnit, S = ONE ? 1 : a.stages;
  const int T = kLanes ? kCta : a.team;
  const int team = kLanes ? 0 : __shfl_sync(0xFFFFFFFFu, threadIdx.x / T, 0);  // the same in a warp, and known to be
  const int t = kLanes ? threadIdx.x : threadIdx.x - team * T;
  const int lanes = kTiles ? a.tiles * 8 : kLanes ? L : T;  // of a row
  const int sub = L ? t / lanes : 0, u = t - sub * lanes;
  // Slot k of a thread is unit u + k * T of its row or, with ROWS, unit u of its
  // row sub + k * R1.  A unit past the row's end works on the row's last one and
  // stores nothing.
  uint32_t eu[NU];  // a unit's first element
#pragma unroll
  for (int k = 0; k < NU; ++k) eu[k] = min(u + k * T, units - 1) * kUnit;
  const int group = R * a.cols;  // elements
  const bool ring_dh = a.dh && a.stage_dh;
  const uint32_t early = early_bytes<XT>(group), late = late_bytes<XT, SAVED>(group, ring_dh);
  const uint32_t weights = smem_u32(smem);
  const uint32_t early0 = weights + weight_bytes(units) + team * S * (early + late), late0 = early0 + S * early;
  uint64_t* const full = bars + team * 3 * kMaxStages;  // [early or late][stage]
  uint64_t* const done = full + 2 * kMaxStages;         // [stage]: each warp has done with the late one
  float* const slot = slots + team * (T >> (kTiles ? 3 : 5)) * NR;
  if (t == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&full[kMaxStages + s], 1);
      mbar_init(&done[s], T >> 5);
    }
    fence_mbar_init();
  }
  __syncthreads();
  chain_wait();
  chain_release();
  const int32_t rows = (int32_t)a.rows, step = gridDim.x * R * (kLanes ? 1 : blockDim.x / T);
  int32_t row0 = (team * gridDim.x + blockIdx.x) * R;
  // One thread of the team: group of rows `from` (64 bits: it may lie past the
  // end, and then nothing is done) into stage s.
  auto fetch_early = [&](int s, int64_t from) {
    if (from >= rows) return;
    const uint64_t policy = policy_evict_first();
    const uint32_t n = (uint32_t)min(rows - (int32_t)from, R) * a.cols, to = early0 + s * early;
    mbar_arrive_expect_tx(&full[s], n * es);
    bulk_g2s(to, static_cast<const char*>(a.dy) + from * a.cols * es, n * es, &full[s], policy);
  };
  auto fetch_late = [&](int s, int64_t from) {
    if (from >= rows) return;
    const uint64_t policy = policy_evict_first();
    const uint32_t n = (uint32_t)min(rows - (int32_t)from, R) * a.cols, to = late0 + s * late;
    uint64_t* bar = &full[kMaxStages + s];
    mbar_arrive_expect_tx(bar, n * ves + (ring_dh ? n * es : 0));
    const char* stream = SAVED ? reinterpret_cast<const char*>(a.codes) : static_cast<const char*>(a.h);
    bulk_g2s(to, stream + from * a.cols * ves, n * ves, bar, policy);
    if (ring_dh) bulk_g2s(to + group * ves, static_cast<const char*>(a.dh) + from * a.cols * es, n * es, bar, policy);
  };
  // With one stage (ONE), the next group's bytes come as far as L2 meanwhile.
  auto ahead = [&](int64_t from) {
    if (from >= rows) return;
    const uint32_t n = (uint32_t)min(rows - (int32_t)from, R) * a.cols;
    const int64_t at = from * a.cols;
    prefetch_l2(static_cast<const char*>(a.dy) + at * es, n * es);
    prefetch_l2((SAVED ? reinterpret_cast<const char*>(a.codes) : static_cast<const char*>(a.h)) + at * ves, n * ves);
    if (a.dh) prefetch_l2(static_cast<const char*>(a.dh) + at * es, n * es);
  };
  if (t == 0) {
    for (int s = 0; s < S; ++s) {
      fetch_early(s, row0 + (int64_t)s * step);
      fetch_late(s, row0 + (int64_t)s * step);
    }
  }
  // The rows' scalars are read one group ahead.
  float next_rstd[NR] = {}, next_scale[U] = {};
  auto scalars = [&](int64_t row) {
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int64_t r = row + (ROWS ? k * R1 : 0);
      if (r >= rows) return;
      if (ROWS || k == 0) next_rstd[ROWS ? k : 0] = a.rstd[r];
      if constexpr (SAVED) next_scale[k] = a.scales[r * a.tiles + eu[ROWS ? 0 : k] / kTile];
    }
  };
  scalars(row0 + sub);
  // The weights in shared memory, in binary32: 16-byte piece p of unit k at p * pieces + 16 * k.
  const uint32_t pieces = weight_bytes(units) / 4;
  {
    Weights w[NU];
#pragma unroll
    for (int j = 0; j < NU; ++j) {
      const int k = threadIdx.x + j * blockDim.x;
      if (k < units) w[j].load(a.weight, a.wt, k);
    }
#pragma unroll
    for (int j = 0; j < NU; ++j) {
      const int k = threadIdx.x + j * blockDim.x;
      float2 f[kPairs];
      w[j].floats(a.wt, f);
      if (k < units) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<float4*>(smem + q * pieces + 16 * k) =
              make_float4(f[2 * q].x, f[2 * q].y, f[2 * q + 1].x, f[2 * q + 1].y);
      }
    }
  }
  __syncthreads();
  float2 acc[NU][kPairs];
#pragma unroll
  for (int k = 0; k < NU; ++k)
#pragma unroll
    for (int i = 0; i < kPairs; ++i) acc[k][i] = both(0.0f);
  bool ok = true;
  const bool second = ROWS || (U > 1 && __any_sync(0xFFFFFFFFu, u + T < units));  // slot, of any lane of the warp
  // The elements of a unit's half that this lane works on first, and second:
  // lanes 4 to 7 of eight begin with the other half, so that the 16-byte reads
  // of eight lanes, 32 bytes apart, cover all banks.
  const uint32_t half0 = threadIdx.x & 4 ? 8 : 0, half1 = 8 - half0;
  int s = 0;
  uint32_t phase = 0, ea = early0, la = late0;  // the stages of this group
  for (int it = 0; row0 < rows; ++it) {
    bool live[NR];
    float rstd[NR], vs[U];
#pragma unroll
    for (int k = 0; k < NR; ++k) {
      live[k] = (L == 0 && k == 0) || ((!kTiles || sub < R1) && (int64_t)row0 + sub + k * R1 < rows);
      rstd[k] = next_rstd[k];
    }
#pragma unroll
    for (int k = 0; k < U; ++k) vs[k] = SAVED ? next_scale[k] * rstd[ROWS ? k : 0] : rstd[ROWS ? k : 0];
    scalars((int64_t)row0 + step + sub);
    if (ONE && t == 0) ahead((int64_t)row0 + step);
    if (ok) ok = mbar_wait_bounded(&full[s], phase) && mbar_wait_bounded(&full[kMaxStages + s], phase);
    if (t == 0 && ok && S > 1 && it > 0) {  // the late stage of the group before
      const int before = s == 0 ? S - 1 : s - 1;
      ok = mbar_wait_bounded(&done[before], s == 0 ? phase ^ 1 : phase);
      if (ok) fetch_late(before, row0 + (int64_t)(S - 1) * step);
    }
    // a row past the end works on the group's first, whose copy is there
    uint32_t at[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int r = ROWS ? k : 0;
      at[k] = (live[r] ? (sub + r * R1) * a.cols : 0) + eu[ROWS ? 0 : k];
    }
    // Half a unit at a time, and the stream's values twice: across the barrier
    // stay the column sums and dy * w.
    float2 g[U][kPairs], d[NR];
#pragma unroll
    for (int k = 0; k < NR; ++k) d[k] = both(0.0f);
#pragma unroll
    for (int j = 0; j < NU; ++j) {
      if (j > 0 && !second) break;
      float2 e[NR];
#pragma unroll
      for (int k = 0; k < NR; ++k) e[k] = both(0.0f);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint32_t h = half ? half1 : half0, wp = weights + h / 4 * pieces + eu[j];
        Unit<XF32> w;
        w.v[2 * half] = lds16(wp);
        w.v[2 * half + 1] = lds16(wp + pieces);
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const int k = ROWS ? r : j;  // the slot
          Unit<XT> dy, v;
          uint2 code;
          dy.take_half(ea + (at[k] + h) * es, half);
          if constexpr (SAVED)
            code = lds8(la + at[k] + h);
          else
            v.take_half(la + (at[k] + h) * es, half);
#pragma unroll
          for (int q = 0; q < kPairs / 2; ++q) {
            const int i = half * (kPairs / 2) + q;
            const float2 x = mul2(SAVED ? e4m3_floats(q < 2 ? code.x : code.y, q) : v.pair(i), both(vs[k]));
            if (live[r]) acc[j][i] = fma2(dy.pair(i), x, acc[j][i]);
            g[k][i] = mul2(dy.pair(i), w.pair(i));
            e[r] = fma2(g[k][i], x, e[r]);
          }
        }
      }
#pragma unroll
      for (int r = 0; r < NR; ++r)
        if (u + j * T < units) d[r] = add2(d[r], e[r]);
    }
    float c[NR];
#pragma unroll
    for (int k = 0; k < NR; ++k) c[k] = d[k].x + d[k].y;
    if constexpr (kLanes) {
#pragma unroll
      for (int k = 0; k < NR; ++k) c[k] = lane_sum<L>(c[k]);
      __syncthreads();
    } else if constexpr (kTiles) {
      tiles_sums(c, slot + (it & 1) * kSlots * NR, team + 1, t, T, a.tiles, sub);
    } else {
      team_sums(c, slot + (it & 1) * kSlots * NR, team + 1, t, T);
    }
    if (t == 0 && ok) fetch_early(s, row0 + (int64_t)S * step);
#pragma unroll
    for (int k = 0; k < NR; ++k) c[k] *= -a.inv_cols * rstd[k];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (k > 0 && !second) break;
      const int r = ROWS ? k : 0, j = ROWS ? 0 : k;
      const bool out = ok && live[r] && u + j * T < units;
      const int64_t to = ((int64_t)row0 + sub + r * R1) * a.cols + (u + j * T) * kUnit;
      Unit<XT> o, v;
      uint2 code;
      o.zero();
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint32_t h = half ? half1 : half0;
        if (ring_dh)
          o.take_half(la + group * ves + (at[k] + h) * es, half);
        else if (a.dh && out)
          o.load_half(static_cast<const char*>(a.dh) + (to + h) * es, half);
        if constexpr (SAVED)
          code = lds8(la + at[k] + h);
        else
          v.take_half(la + (at[k] + h) * es, half);
#pragma unroll
        for (int q = 0; q < kPairs / 2; ++q) {
          const int i = half * (kPairs / 2) + q;
          const float2 x = SAVED ? e4m3_floats(q < 2 ? code.x : code.y, q) : v.pair(i);
          const float2 f = both(c[r] * vs[k]);
          // FP32: dh, mostly the largest term, is added last and rounded once; a 16-bit result hides the
          // rounding that one instruction less costs.
          if constexpr (XT == XF32)
            o.set_pair(i, add2(fma2(g[k][i], both(rstd[r]), mul2(x, f)), o.pair(i)));
          else
            o.set_pair(i, fma2(g[k][i], both(rstd[r]), fma2(x, f, o.pair(i))));
        }
        if (out) o.store_half(static_cast<char*>(a.dx) + (to + h) * es, half);
      }
    }
    __syncwarp();
    if ((t & 31) == 0) mbar_arrive(&done[s]);
    if (t == 0 && ok && S == 1) {
      ok = mbar_wait_bounded(&done[0], phase);
      if (ok) fetch_late(0, row0 + (int64_t)step);
    }
    if ((int64_t)row0 + step >= rows) break;  // before the sum could pass 32 bits
    row0 += step;
    ea += early, la += late;
    if (++s == S) s = 0, phase ^= 1, ea = early0, la = late0;
  }
  if (!ok) atomicAdd(&g_norm_wait_failures, 1u);
  if (!ok && t == 0) {
    // Copies may still be on their way.
    for (int j = 0; j < 2 * kMaxStages; ++j)
      if (j % kMaxStages < S) mbar_drain(&full[j]);
  }
  __syncthreads();  // the rings are free: every team has done with its last row
  float* fold = reinterpret_cast<float*>(smem);  // [team or sub-row][columns]
  const int width = kLanes ? L * kUnit : a.cols, deep = kLanes ? R1 : blockDim.x / T * R1;
#pragma unroll
  for (int k = 0; k < NU; ++k) {
    if (!kLanes && (u + k * T >= units || sub >= R1)) break;
    float* f = fold + (team * R1 + sub) * width + (u + k * T) * kUnit;
#pragma unroll
    for (int i = 0; i < kPairs; i += 2)
      *reinterpret_cast<float4*>(f + (i < kPairs / 2 ? half0 : half1) + 2 * i % 8) =
          make_float4(acc[k][i].x, acc[k][i].y, acc[k][i + 1].x, acc[k][i + 1].y);
  }
  __syncthreads();
  for (int col = 4 * threadIdx.x; col < a.cols; col += 4 * blockDim.x) {
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int j = 0; j < deep; ++j) {
      const float4 x = *reinterpret_cast<const float4*>(fold + j * width + col);
      v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
    }
    *reinterpret_cast<float4*>(a.parts + (int64_t)blockIdx.x * a.cols + col) = v;
  }
}

// dweight[col] = sum over the partial rows: 32 columns a CTA, 16 warps that each
// sum every 16th partial row, joined in a fixed order.
constexpr int kFoldWarps = 16, kFoldLoads = 20;
__global__ __launch_bounds__(32 * kFoldWarps, 4) void k_norm_dweight(const float* parts, int32_t nparts, int32_t cols,
                                                                     void* dweight, int32_t dt) {
  __shared__ float s[kFoldWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  chain_wait();
  chain_release();
  float v = 0.0f;
  if (col < cols) {
    const float* at = parts + (int64_t)warp * cols + col;
    for (int p = warp; p < nparts; p += kFoldWarps * kFoldLoads) {
      float x[kFoldLoads];  // all in flight at once
#pragma unroll
      for (int j = 0; j < kFoldLoads; ++j) {
        x[j] = p + j * kFoldWarps < nparts ? *at : 0.0f;
        at += (int64_t)kFoldWarps * cols;
      }
#pragma unroll
      for (int j = 0; j < kFoldLoads; ++j) v += x[j];
    }
  }
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

template <int XT, bool SAVED, int L, int U, bool ROWS>
mp_status launch_bwd_rows(NormBwd a, const RowShape& s, int* parts, cudaStream_t st) {
  static std::atomic<uint64_t> opted[2] = {0, 0};
  constexpr bool kLanes = L > kInTiles;
  const int rows_per_group = (L == kInTiles ? a.group : s.rows_per_cta) * (ROWS ? U : 1);
  const int64_t groups = (a.rows + rows_per_group - 1) / rows_per_group;
  const int weights = weight_bytes(a.cols / kUnit), elements = rows_per_group * a.cols;
  const int early = early_bytes<XT>(elements);
  // FP32 rows of over 14336 without a checkpoint do not fit with dh, which is then read directly.
  a.stage_dh = a.dh && early + late_bytes<XT, SAVED>(elements, true) + weights <= kSmemBytes;
  const int bytes = early + late_bytes<XT, SAVED>(elements, a.stage_dh);  // with the weights at most 224 KB
  // Rows in lanes: as many CTAs on an SM as registers allow.  Rows of whole
  // teams: one CTA of as many teams, but of no more than spread the rows over
  // all SMs.  Either so many that each has two stages; then as many stages, up
  // to kMaxStages, as there is room.
  const int team = kLanes ? kCta : L == kInTiles ? (a.group * a.tiles + 3) / 4 * 32 : team_of(s, ROWS ? 1 : U);
  int per_sm = (U == 1 ? 1024 : ROWS ? kRowsThreads : 512) / team;  // threads of 64, 96 and 128 registers on an SM
  if (!kLanes && per_sm > kMaxTeams) per_sm = kMaxTeams;
  while (per_sm > 1 && (kLanes ? (2 * bytes + weights) * per_sm > kSmemShared : 2 * bytes * per_sm + weights > kSmemBytes))
    --per_sm;
  const int64_t spread = (groups + sm_count() - 1) / sm_count();
  const int teams = kLanes ? 1 : (int)(per_sm < spread ? per_sm : spread);
  a.team = team;
  a.stages = ((kLanes ? kSmemShared / per_sm : kSmemBytes) - weights) / (bytes * teams);
  if (a.stages > kMaxStages) a.stages = kMaxStages;
  int smem = weights + teams * a.stages * bytes;
  const int fold = (kLanes ? kCta * kUnit : teams * (L == kInTiles ? a.group : 1) * a.cols) * 4;  // the join of the column sums
  if (smem < fold) smem = fold;
  const bool one = a.stages == 1;  // only rows of whole teams and two units a thread are that long
  const auto kernel = one ? k_norm_bwd<XT, SAVED, L, U, ROWS, L == 0 && U == 2 && !ROWS>
                          : k_norm_bwd<XT, SAVED, L, U, ROWS, false>;
  if (!smem_ok(kernel, smem, opted[one])) return MP_ECUDA;
  const int grid = resident_grid((groups + teams - 1) / teams, kLanes ? per_sm : 1);
  const int64_t room = parts_of(a.rows, a.cols);  // partial rows in the workspace
  *parts = (int)(grid < room ? grid : room);
  launch_chained(kernel, dim3(*parts), dim3(teams * team), smem, st, a);
  note_launches(1);
  return launch_status();
}

// The row length, in threads of one unit, up to which a team takes two rows at a
// time instead of two units of one.  Two rows need more of shared memory for each
// team, so that of long rows fewer are in flight.  GPU time in us, with two rows
// and with two units: BF16 from the checkpoint [16384 x 1040] 28.1 and 33.7,
// [8192 x 2560] 29.6 and 30.6, [8192 x 3072] 34.2 and 34.0, [8192 x 4096] 38.1 and
// 40.2, [16384 x 5120] 93.0 and 92.0, [4096 x 8192] 41.9 and 40.4; F32 [4096 x 1040]
// 14.2 and 15.8, [16384 x 1536] 62.3 and 63.0, [4096 x 2048] 23.9 and 22.7,
// [16384 x 2560] 108.7 and 98.7.
// BF16 from the stream, whose stage is a fifth larger: from 2048 to 3072 columns an
// SM then holds one team fewer, and two rows are still as fast or faster.  [16384 x
// 2048] 46.7 and 47.7, [8192 x 2304] 28.4 and 30.6, [8192 x 2560] 30.8 and 32.1,
// [8192 x 3072] 37.2 and 37.2, [8192 x 3584] 40.8 and 41.8, [8192 x 4096] 45.6 and
// 47.0, [16384 x 5120] 113.8 and 104.0; without dh 38.9 and 40.0 at 2048 columns,
// 26.5 and 28.0 at 2560, 30.9 and 31.6 at 3072, but 40.8 and 39.8 at 4096.  F32 from
// the stream [4096 x 1040] 16.3 and 18.1, [16384 x 1536] 63.6 and 64.7.
template <int XT>
constexpr int two_rows_up_to() { return XT == XF32 ? 96 : 256; }

// Rows (of 5 to 16 tiles) that would leave a sixth of whole warps idle lie in
// tiles of a team that takes twice `group` of them.  GPU time in us over inputs
// beyond L2 with this layout and without, BF16 from the checkpoint: [4096 x 640] 8.3
// and 10.7, [16384 x 528] 18.0 and 22.9, [16384 x 576] 18.4 and 22.4, [16384 x 768]
// 21.4 and 22.5, [16384 x 1040] 26.1 and 29.2, [16384 x 1280] 30.1 and 30.1, [16384 x
// 1664] 35.9 and 36.8; where fewer lanes are idle it lost ([16384 x 896] 22.9 and
// 22.0, [16384 x 1792] 37.7 and 36.0).
// From the stream: [16384 x 528] 18.0 and 23.0, [4096 x 640] 10.5 and 11.2, [16384 x
// 768] 22.9 and 23.7, [16384 x 1040] 27.6 and 30.7, [16384 x 1280] 32.8 and 33.3,
// [16384 x 1664] 40.3 and 41.0.
// FP32 was as often slower as faster ([16384 x 640] 31.1 and 29.6, [16384 x 576]
// 25.0 and 29.3).
bool tiles_save_lanes(int tiles) { return tiles > 4 && tiles <= kTilesMax && 6 * tiles <= 5 * ((tiles + 3) / 4 * 4); }
// Such rows of a team, for each of a thread's two: as many as let the most be on
// an SM, by its registers and by shared memory for two stages of `bytes` each.
int rows_of_team(const NormBwd& a, int bytes) {
  int best = 1, most = 0;
  for (int rows = 1; rows <= 4; ++rows) {
    const int by_regs = kRowsThreads / 32 / ((rows * a.tiles + 3) / 4);
    const int by_smem = (kSmemBytes - weight_bytes(a.cols / kUnit)) / (2 * rows * bytes);
    int teams = by_regs < by_smem ? by_regs : by_smem;
    if (teams > kMaxTeams) teams = kMaxTeams;
    if (teams * rows > most) most = teams * rows, best = rows;
  }
  return best;
}

template <int XT, bool SAVED>
mp_status launch_bwd(NormBwd a, void* dweight, int32_t dt, cudaStream_t st) {
  int parts = 0;
  if (a.rows > 0) {
    const RowShape s = row_shape(a.cols);
    mp_status r;
    if (XT != XF32 && tiles_save_lanes(a.tiles)) {
      a.group = rows_of_team(a, 2 * (early_bytes<XT>(a.cols) + late_bytes<XT, SAVED>(a.cols, a.dh)));
      r = launch_bwd_rows<XT, SAVED, XT == XF32 ? 0 : kInTiles, 2, true>(a, s, &parts, st);
    } else {
      r = s.lanes == 8    ? launch_bwd_rows<XT, SAVED, 8, 1, false>(a, s, &parts, st)
          : s.lanes == 16 ? launch_bwd_rows<XT, SAVED, 16, 1, false>(a, s, &parts, st)
          : s.lanes == 32 ? launch_bwd_rows<XT, SAVED, 32, 1, false>(a, s, &parts, st)
          : s.threads <= two_rows_up_to<XT>() ? launch_bwd_rows<XT, SAVED, 0, 2, true>(a, s, &parts, st)
                                              : launch_bwd_rows<XT, SAVED, 0, 2, false>(a, s, &parts, st);
    }
    if (r != MP_OK) return r;
  }
  launch_chained(k_norm_dweight, dim3((a.cols + 31) / 32), dim3(32 * kFoldWarps), 0, st, (const float*)a.parts,
                 (int32_t)parts, a.cols, dweight, dt);
  note_launches(1);
  return launch_status();
}

bool float_type(mp_dtype t) { return t == MP_F32 || t == MP_F16 || t == MP_BF16; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace

uint32_t norm_wait_failures() {
  uint32_t v = 0;
  if (cudaMemcpyFromSymbol(&v, g_norm_wait_failures, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
  return v;
}

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
  if (rows > kMaxRows || cols > kMaxCols || cols % (scale_block == 32 ? 32 : 16) != 0) return MP_ESHAPE;
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
  a.ckpt = static_cast<uint8_t*>(ckpt), a.ckpt_scales = ckpt_scales;
  a.rows = rows, a.cols = (int32_t)cols, a.tiles = tiles, a.wt = w_dtype, a.eps = eps, a.inv_cols = 1.0f / (float)cols;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (x_dtype) {
    case MP_F32: return launch_fwd_type<XF32>(a, st);
    case MP_F16: return launch_fwd_type<XF16>(a, st);
    default: return launch_fwd_type<XBF16>(a, st);
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
  if (rows > kMaxRows || cols > kMaxCols || cols % 16 != 0) return MP_ESHAPE;
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
  a.inv_cols = 1.0f / (float)cols;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (x_dtype) {
    case MP_F32: return ckpt ? launch_bwd<XF32, true>(a, dweight, dw_dtype, st) : launch_bwd<XF32, false>(a, dweight, dw_dtype, st);
    case MP_F16: return ckpt ? launch_bwd<XF16, true>(a, dweight, dw_dtype, st) : launch_bwd<XF16, false>(a, dweight, dw_dtype, st);
    default: return ckpt ? launch_bwd<XBF16, true>(a, dweight, dw_dtype, st) : launch_bwd<XBF16, false>(a, dweight, dw_dtype, st);
  }
}
