// mp_ffn_few.cu — the gated feed-forward products for few rows (few_forward): a decoding
// step, or the backward pass of a short sequence.
//
// The weights are read once and everything else is small, so the weights are
// the operand with 128 rows (of M = 128 matrix instructions) and x is the other
// one, padded to 16, 32, 64 or 128 columns.  A cluster of up to eight CTAs
// shares a tile of 128 hidden elements (both matrices' rows of them), each
// with a part of the contraction, whose runs are added in registers as they end;
// the parts' sums meet in shared memory and are added in the order of the parts, a
// few rows of x for each CTA.  dx is the same with tiles of 128 columns of the
// weights, taken as they lie (MN-major).
//
// Bound by DRAM: the stages of the CTAs on an SM, some 200 KB, are its bytes in
// flight.  One row of 4096 x 14336 BF16: 38 us, 0.92 of the copy rate; 64 rows 42;
// 128 rows 46; dx of one row 38.  What is left is the chain before the
// first tile and after the last: sums to shared memory, the cluster's barrier,
// the other CTAs' sums.
#include "mp_chain.cuh"
#include "mp_ffn.cuh"

namespace mp {
namespace {

constexpr int kTileRows = 128;                       // of a matrix instruction
constexpr int kWeightBytes = kTileRows * kBlockK * 2;  // one matrix's part of a stage
constexpr int kResultWarps = 8;
constexpr int kThreads = (kResultWarps + 2) * 32;    // one more warp copies, another issues
constexpr int kBarrierBytes = 256;

// Columns N of x's operand, matrices in a tile: two (FWD, AGAIN) or one (STORE).
template <int N, int EP>
struct Shape {
  static constexpr int kMatrices = EP == STORE ? 1 : 2;
  static constexpr int kXBytes = N * kBlockK * 2;
  static constexpr int kStageBytes = kMatrices * kWeightBytes + kXBytes;
  static constexpr int kSumBytes = N * kMatrices * kTileRows * 4;
  // Two CTAs an SM have 113 KB each: two stages of 64 or more columns and two
  // matrices, and then one CTA with five is faster (1024 x 2816 for 64 rows 7.3
  // us instead of 11.3).
  static constexpr int kCtas = kMatrices == 2 && N >= 64 ? 1 : 2;
  static constexpr int kStages = ((kCtas == 2 ? 113 : 226) * 1024 - kBarrierBytes) / kStageBytes;
  static constexpr int kRing = kStages * kStageBytes;
  static constexpr int kSmem = (kRing > kSumBytes ? kRing : kSumBytes) + kBarrierBytes;
  // Runs of the contraction take turns in places of their own in TMEM: one is
  // added to registers while the next is formed.
  static constexpr int kRunColumns = kMatrices * N;
  static constexpr int kColumns = 512 / kCtas;
  static constexpr int kPlaces = kColumns / kRunColumns < 8 ? kColumns / kRunColumns : 8;
  static constexpr int kGroups = kRunColumns < 32 ? 1 : kRunColumns / 32;  // of 16 columns, in a result thread
  static_assert(kStages >= 2 && kPlaces >= 2 && kSumBytes <= 128 * 1024, "stages, TMEM columns");
  static_assert((2 * kStages + 2 * kPlaces) * 8 + 4 <= kBarrierBytes, "barriers and the TMEM address");
};

struct Few {
  CUtensorMap w[2], x[2];  // weights; x, or dg and du
  int32_t parts, run;      // CTAs of a cluster; stages of a run
  int32_t blocks0, blocks;  // stages of the first operand pair (STORE), and in all
  int32_t rows, cols;      // rows of x; columns of the result
  FfnOut o;
};

__device__ unsigned int g_few_wait_failures;  // bounded waits that gave up (read by mp_wait_failures)

__device__ __forceinline__ void tma_load(uint32_t dst, const void* map, int32_t x, int32_t y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}

// Four values of a row in each lane.
struct Four {
  float2 a, b;
};
__device__ __forceinline__ uint32_t amax4(const Four& v) {
  const float m = max3_abs_nan(0.0f, v.a.x, v.a.y);
  return __float_as_uint(max3_abs_nan(m, v.b.x, v.b.y));
}
__device__ __forceinline__ uint32_t nonfinite_code(float v) {
  return (fabsf(v) < INFINITY ? 0u : 0x7Fu) | ((__float_as_uint(v) >> 24) & 0x80u);
}
__device__ __forceinline__ uint32_t codes4(const Four& v, uint32_t m, float mul, bool e5m2, bool mx) {
  if (__builtin_expect(m >= kInfBits, 0))
    return mx ? 0u
              : nonfinite_code(v.a.x) | nonfinite_code(v.a.y) << 8 | nonfinite_code(v.b.x) << 16 |
                    nonfinite_code(v.b.y) << 24;
  const float2 a = mul2(v.a, both(mul)), b = mul2(v.b, both(mul));
  return e5m2 ? cvt_e5m2x2(a.x, a.y) | cvt_e5m2x2(b.x, b.y) << 16 : cvt_e4m3x2(a.x, a.y) | cvt_e4m3x2(b.x, b.y) << 16;
}
template <bool BF16>
__device__ __forceinline__ void store16(void* base, int64_t at, const Four& v) {
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(base) + at) = make_uint2(pack16<BF16>(v.a), pack16<BF16>(v.b));
}

// A row's results: 128 columns from col0, four in each lane; `in`: they are in the matrix.
template <bool BF16, int EP>
__device__ __forceinline__ void finish_row(const Few& f, int row, int tile, int col, bool in, Four g, Four u) {
  const FfnOut& o = f.o;
  const int64_t at = (int64_t)row * f.cols + col;
  const int lane = threadIdx.x & 31;
  if constexpr (EP == STORE) {
    if (in) store16<BF16>(o.p, at, g);
  } else if constexpr (EP == AGAIN) {
    if (!in) return;
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(o.dp) + at);
    Four dg, du;
    slopes(pair16<BF16>(w.x), g.a, u.a, &dg.a, &du.a);
    slopes(pair16<BF16>(w.y), g.b, u.b, &dg.b, &du.b);
    store16<BF16>(o.dg, at, dg);
    store16<BF16>(o.du, at, du);
  } else {
    if (o.gate && in) {
      store16<BF16>(o.gate, row * o.ld + col, g);
      store16<BF16>(o.up, row * o.ld + col, u);
    }
    if (o.ckpt) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const Four& v = j ? u : g;
        const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, in ? amax4(v) : 0u);
        float mul;
        const float scale = tile_scale(m, 448.0f, &mul);
        if (lane == 0) o.ckpt_scales[((int64_t)j * f.rows + row) * o.tiles + tile] = scale;
        if (in) *reinterpret_cast<uint32_t*>(o.ckpt + (int64_t)j * f.rows * f.cols + at) = codes4(v, m, mul, false, false);
      }
    }
    const Four p{gated(g.a, u.a), gated(g.b, u.b)};
    if constexpr (EP == FWD16) {
      if (in) store16<BF16>(o.p, at, p);
    } else {
      uint32_t m = in ? amax4(p) : 0u;
      float mul;
      if (o.mx) {
        m = tile_max(m);  // over the eight lanes of a 1x32 block
        uint32_t byte;
        mx_scale(m, o.e5m2 ? 15u : 8u, &mul, &byte);
        if ((lane & 7) == 0 && in) static_cast<uint8_t*>(o.p_scales)[(int64_t)row * o.per_row + (col >> 5)] = (uint8_t)byte;
      } else {
        m = __reduce_max_sync(0xFFFFFFFFu, m);
        const float scale = tile_scale(m, o.e5m2 ? 57344.0f : 448.0f, &mul);
        if (lane == 0) static_cast<float*>(o.p_scales)[(int64_t)row * o.per_row + tile] = scale;
      }
      if (in) *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(o.p) + at) = codes4(p, m, mul, o.e5m2, o.mx);
    }
  }
}

template <bool BF16, int N, int EP>
__global__ __launch_bounds__(kThreads, Shape<N, EP>::kCtas) void k_ffn_few(const __grid_constant__ Few f) {
  using S = Shape<N, EP>;
  extern __shared__ __align__(1024) unsigned char smem[];
  uint64_t* const full = reinterpret_cast<uint64_t*>(smem + S::kSmem - kBarrierBytes);
  uint64_t *const empty = full + S::kStages, *const done = empty + S::kStages, *const free = done + S::kPlaces;
  uint32_t* const tmem_at = reinterpret_cast<uint32_t*>(free + S::kPlaces);
  float* const sums = reinterpret_cast<float*>(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = blockIdx.x % f.parts, tile = blockIdx.x / f.parts;
  const int k0 = (int)((int64_t)f.blocks * part / f.parts), k1 = (int)((int64_t)f.blocks * (part + 1) / f.parts);

  if (warp == kResultWarps && lane == 0) {
    for (int s = 0; s < S::kStages; ++s) mbar_init(full + s, 1), mbar_init(empty + s, 1);
    for (int b = 0; b < S::kPlaces; ++b) mbar_init(done + b, 1), mbar_init(free + b, kResultWarps);
    fence_mbar_init();
  }
  if (warp == 0 && lane < 2) prefetch_tensor_map(f.w + lane);
  if (warp == 1 && lane < (EP == STORE ? 2 : 1)) prefetch_tensor_map(f.x + lane);
  __syncthreads();
  chain_wait();

  // An SM has room for other kernels beside this one, and tensor memory has to be
  // waited for where they hold it.  So this CTA waits for nobody while it holds
  // some itself: not for the kernel before (it is allocated after that), nor for
  // the cluster (freed before its barriers); and the next kernel is let in when
  // this one has got its own.  The first tiles are on their way meanwhile.
  bool ok = true;
  if (warp == kResultWarps) {
    if (lane == 0) {
      for (int kb = k0, it = 0; kb < k1; ++kb, ++it) {
        const int s = it % S::kStages;
        if (!(ok = mbar_wait_bounded(empty + s, ((it / S::kStages) & 1) ^ 1))) break;
        mbar_arrive_expect_tx(full + s, S::kStageBytes);
        const uint32_t to = smem_u32(smem + s * S::kStageBytes);
        if constexpr (EP == STORE) {
          const int second = kb >= f.blocks0, k = (second ? kb - f.blocks0 : kb) * kBlockK;
          tma_load(to, f.w + second, tile * kTileRows, k, full + s);
          tma_load(to + kMnBlockBytes, f.w + second, tile * kTileRows + 64, k, full + s);
          tma_load(to + kWeightBytes, f.x + second, k, 0, full + s);
        } else {
          tma_load(to, f.w, kb * kBlockK, tile * kTileRows, full + s);
          tma_load(to + kWeightBytes, f.w + 1, kb * kBlockK, tile * kTileRows, full + s);
          tma_load(to + 2 * kWeightBytes, f.x, kb * kBlockK, 0, full + s);
        }
      }
    }
  } else if (warp == kResultWarps + 1) {
    tmem_alloc<1>(smem_u32(tmem_at), S::kColumns);
    chain_release();
    __syncwarp();
    asm volatile("bar.arrive 1, %0;" ::"n"((kResultWarps + 1) * 32) : "memory");
    const uint32_t tmem = *tmem_at;
    if (lane == 0) {
      constexpr bool MN = EP == STORE;
      constexpr uint32_t idesc = instr_desc<BF16, MN, false>(kTileRows, N);
      int r = -1;  // the run
      for (int kb = k0, it = 0, left = 0; kb < k1; ++kb, ++it, --left) {  // left: its stages to come
        if (left == 0) {
          left = f.run, ++r;
          if (!(ok = mbar_wait_bounded(free + r % S::kPlaces, ((r / S::kPlaces) & 1) ^ 1))) break;
        }
        const int s = it % S::kStages;
        if (!(ok = mbar_wait_bounded(full + s, (it / S::kStages) & 1))) break;
        tmem_fence_after();
        const uint32_t at = smem_u32(smem + s * S::kStageBytes);
        const uint64_t x = operand_desc<false>(at + S::kMatrices * kWeightBytes);
        const uint32_t d = tmem + r % S::kPlaces * S::kRunColumns;
#pragma unroll
        for (int m = 0; m < S::kMatrices; ++m) {
          const uint64_t w = operand_desc<MN>(at + m * kWeightBytes);
#pragma unroll
          for (int j = 0; j < kBlockK / 16; ++j)
            mma_f16<1>(d + m * N, w + j * kDescStep<MN>, x + j * kDescStep<false>, idesc, left != f.run || j != 0);
        }
        mma_commit<1>(empty + s);
        if (left == 1 || kb == k1 - 1) mma_commit<1>(done + r % S::kPlaces);
      }
      // No instruction is left at work on shared or tensor memory, also where the
      // warps that read the results have given up.
      if (ok) ok = mbar_wait_bounded(done + r % S::kPlaces, (r / S::kPlaces) & 1);
      if (!ok)
        for (int s = 0; s < S::kStages; ++s) mbar_drain(full + s);
    }
  } else {
    named_barrier(1, (kResultWarps + 1) * 32);  // tensor memory is there
    const uint32_t tmem = *tmem_at;
    const int quad = warp & 3;  // the lanes that a warp can read
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    const int runs = (k1 - k0 + f.run - 1) / f.run;
    // The warp's columns of a run, 16 at a time; those without a row of x stay out.
    const auto column = [&](int i) { return (2 * i + (warp >> 2)) * 16; };
    const auto used = [&](int c) { return c < S::kRunColumns && c % N < f.rows; };
    // Waits for a run's sums; where they are.
    const auto run_done = [&](int r) {
      const int place = r % S::kPlaces;
      ok = ok && __all_sync(0xFFFFFFFFu, mbar_wait_bounded(done + place, (r / S::kPlaces) & 1));
      tmem_fence_after();
      return lanes + place * S::kRunColumns;
    };
    const auto run_read = [&](int r) {  // their place is free
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(free + r % S::kPlaces);
    };
    uint32_t acc[S::kGroups][16];
    uint32_t from = run_done(0);
#pragma unroll
    for (int i = 0; i < S::kGroups; ++i)
      if (used(column(i))) tmem_load16(acc[i], from + column(i));
    tmem_wait();
#pragma unroll
    for (int i = 0; i < S::kGroups; ++i) loaded(acc[i]);
    run_read(0);
    for (int r = 1; r < runs; ++r) {
      from = run_done(r);
#pragma unroll
      for (int i = 0; i < S::kGroups; ++i) {
        if (!used(column(i))) continue;
        uint32_t v[16];
        tmem_load16(v, from + column(i));
        tmem_wait();
        loaded(v);
#pragma unroll
        for (int k = 0; k < 16; ++k) acc[i][k] = __float_as_uint(__uint_as_float(acc[i][k]) + __uint_as_float(v[k]));
      }
      run_read(r);
    }
    // This part's sums: [row of x][matrix][128], where the ring was.
#pragma unroll
    for (int i = 0; i < S::kGroups; ++i) {
      const int c = column(i);
      if (!used(c)) continue;
#pragma unroll
      for (int k = 0; k < 16; ++k)
        sums[((c % N + k) * S::kMatrices + c / N) * kTileRows + quad * 32 + lane] = __uint_as_float(acc[i][k]);
    }
    tmem_fence_before();
  }
  __syncthreads();
  tmem_fence_after();
  if (warp < kResultWarps && !ok)  // sums that are not complete, now that no copy is on its way to the ring
    for (int i = threadIdx.x; i < S::kSumBytes / 4; i += kResultWarps * 32) sums[i] = __uint_as_float(complete_or_nan(ok, 0));
  if (warp == kResultWarps + 1) tmem_free<1>(*tmem_at, S::kColumns);
  __syncwarp();
  cluster_sync();  // every part's sums stand
  if (warp < kResultWarps) {
    const int col = tile * kTileRows + lane * 4;
    const bool in = col < f.cols;
    const uint32_t from = smem_u32(sums) + lane * 16;
    for (int row = part + warp * f.parts; row < f.rows; row += kResultWarps * f.parts) {
      Four v[S::kMatrices];
#pragma unroll
      for (int m = 0; m < S::kMatrices; ++m) v[m].a = v[m].b = both(0.0f);
      for (int p = 0; p < f.parts; ++p) {
        const uint32_t at = map_rank(from, p) + row * S::kMatrices * kTileRows * 4;
#pragma unroll
        for (int m = 0; m < S::kMatrices; ++m) {
          const float4 q = ld_cluster(at + m * kTileRows * 4);
          v[m].a = add2(v[m].a, make_float2(q.x, q.y));
          v[m].b = add2(v[m].b, make_float2(q.z, q.w));
        }
      }
      finish_row<BF16, EP>(f, row, tile, col, in, v[0], v[S::kMatrices - 1]);
    }
  }
  if (!ok) atomicAdd(&g_few_wait_failures, 1u);
  cluster_sync();  // no CTA leaves while another reads its sums
}

template <bool BF16, int N, int EP>
mp_status launch(Few& f, int tiles, cudaStream_t st) {
  using S = Shape<N, EP>;
  static std::atomic<uint64_t> done{0};
  const auto kernel = k_ffn_few<BF16, N, EP>;
  if (!smem_opt_in(kernel, S::kSmem, done)) return MP_ECUDA;
  // As many parts, by twos, as there is place for at once, each with two stages
  // at least: clusters of 3, 5, 6 and 7 leave places empty where two CTAs share an SM
  // (2048 x 5504 for one row: four parts 11.0 us, seven 16.1).  Where a CTA has its
  // SM alone they go either way: three parts for two take 100 rows of 2048 x 5504
  // from 15.7 to 14.8 us and 64 rows from 13.6 to 13.5, six for four 64 rows of 1024 x
  // 2816 from 7.4 to 8.4.  A second wave costs as much (4096 x 14336: two parts 38 us,
  // four 40).
  f.parts = 1;
  while (f.parts < 8 && tiles * f.parts * 2 <= sm_count() * S::kCtas && f.blocks >= 4 * f.parts) f.parts *= 2;
  const int most = ceil_div(f.blocks, f.parts);  // stages of a part
  f.run = ceil_div(most, ceil_div(most, run_of<EP>(f.o)));  // runs of one length
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = f.parts, attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(tiles * f.parts);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, kernel, f) != cudaSuccess) {
    cudaGetLastError();
    return MP_ECUDA;
  }
  note_launches(1);
  return MP_OK;
}

template <bool BF16, int EP>
mp_status by_rows(Few& f, int tiles, cudaStream_t st) {
  if (f.rows <= 16) return launch<BF16, 16, EP>(f, tiles, st);
  if (f.rows <= 32) return launch<BF16, 32, EP>(f, tiles, st);
  if (EP == STORE || f.rows <= 64) return launch<BF16, 64, EP>(f, tiles, st);  // dx: kFewDxRows
  if constexpr (EP != STORE) return launch<BF16, 128, EP>(f, tiles, st);
}
template <int EP>
mp_status by_type(bool bf16, Few& f, int tiles, cudaStream_t st) {
  return bf16 ? by_rows<true, EP>(f, tiles, st) : by_rows<false, EP>(f, tiles, st);
}
int columns_of(int64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128; }

}  // namespace

mp_status ffn_few_project(int ep, bool bf16, const void* x, const void* w_gate, const void* w_up, int64_t rows,
                          int64_t width, int64_t hidden, const FfnOut& out, cudaStream_t st) {
  Few f;
  if (!map16(&f.x[0], x, rows, width, width, columns_of(rows)) || !map16(&f.w[0], w_gate, hidden, width, width, kTileRows) ||
      !map16(&f.w[1], w_up, hidden, width, width, kTileRows))
    return MP_ECUDA;
  f.o = out;
  f.blocks = f.blocks0 = ceil_div(width, kBlockK);
  f.rows = (int32_t)rows, f.cols = (int32_t)hidden;
  const int tiles = ceil_div(hidden, kTileRows);
  return ep == FWD16 ? by_type<FWD16>(bf16, f, tiles, st)
         : ep == FWD8 ? by_type<FWD8>(bf16, f, tiles, st) : by_type<AGAIN>(bf16, f, tiles, st);
}

mp_status ffn_few_dx(bool bf16, const void* dg, const void* du, const void* w_gate, const void* w_up, int64_t rows,
                     int64_t width, int64_t hidden, void* dx, cudaStream_t st) {
  Few f;
  const int n = columns_of(rows);
  if (!map16(&f.x[0], dg, rows, hidden, hidden, n) || !map16(&f.x[1], du, rows, hidden, hidden, n) ||
      !map16(&f.w[0], w_gate, hidden, width, width, 64) || !map16(&f.w[1], w_up, hidden, width, width, 64))
    return MP_ECUDA;
  f.o = FfnOut{};
  f.o.p = dx;
  f.blocks0 = ceil_div(hidden, kBlockK), f.blocks = 2 * f.blocks0;
  f.rows = (int32_t)rows, f.cols = (int32_t)width;
  return by_type<STORE>(bf16, f, ceil_div(width, kTileRows), st);
}

uint32_t ffn_few_wait_failures() {
  uint32_t v = 0;
  if (cudaMemcpyFromSymbol(&v, g_few_wait_failures, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
  return v;
}

}  // namespace mp
