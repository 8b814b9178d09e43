// mp_ffn.cu — the gated feed-forward block's matrix products: both projections
// with the SwiGLU product formed on them in one kernel, and their backward pass.
//
// Forward: g = x Wg^T, u = x Wu^T, p = (g * s(g)) * u; g and u never reach
// memory unless asked for.  Backward, with g and u as saved (16 bits, or the
// 8-bit checkpoint) or formed again from x by the forward kernel's main loop:
//   dg = dp * u * (s + g * s * (1 - s)),  du = dp * g * s,
//   dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x.
// dg and du go through a 16-bit workspace: they are the operands of 16-bit
// matrix instructions, which is the one rounding inside the backward pass.
//
// One kernel does all of it: 256 x 256 tiles of a product on pairs of CTAs
// (tcgen05, 128 rows of the tile in each CTA's TMEM), persistent, with roles by
// warp: two copy operand tiles (TMA, six stages of 64 steps of the contraction),
// one issues the matrix instructions, eight form the results.  The forward
// tile's 256 columns are 128 of g and the same 128 of u: the pair's first CTA
// holds the gate weights' half of the operand and the second the up weights', so
// the thread that has an element of g has that of u.  Backward, dx and the
// weights' gradients are one launch, so that no pair waits between them.
//
// Sums: the tensor core adds to its binary32 accumulator by truncation, which
// over a contraction of 4096 leaves results 4e-6 too small.  So after every run
// of stages the sums so far leave TMEM and are added to registers with correct
// rounding, while the next run goes into the other half of TMEM.
//
// Bound by the tensor pipe, which is active 89 % of the cycles of [2048 x 4096 x
// 14336], and in a warm loop by the power limit: [8192 x 4096 x 14336] BF16
// forward 945 to 970 us cold and 1075 warm (the library product of the same shape
// without the activation 1052 and 1085), with an FP8 product and the 8-bit
// checkpoint 990 to 1025 and 1148, with the checkpoint beside a 16-bit product 1000
// to 1020 cold, since their runs are shorter; dx and the weights' gradients 2250 and
// 2320 to 2450 (2161 and 2254).  Small products are a chain of latencies:
// 12,600 cycles for one tile, half of them before and after its work.
#include <type_traits>

#include "mp_chain.cuh"
#include "mp_ffn.cuh"

namespace mp {
namespace {

constexpr int kHalf = 128;         // rows of a tile in one CTA
constexpr int kOperandBytes = kHalf * kBlockK * 2;
constexpr int kResultWarps = 8;
constexpr int kRingBytes = 192 * 1024;
constexpr int kStagingBytes = 4096;  // 32 rows of 128 bytes, for each of those warps
// Three warpgroups: two form results, with 128 sums a thread, one copies and
// issues.  384 threads start with 168 registers each; the split adds up to that.
constexpr int kThreads = (kResultWarps + 4) * 32;
constexpr int kResultRegisters = 224, kOtherRegisters = 56;
static_assert(kResultWarps * kResultRegisters + 4 * kOtherRegisters <= (kResultWarps + 4) * 168, "registers of a CTA");
// A tile has W = 256 columns, or 128 where there are few tiles.
template <int W>
struct Wide {
  static constexpr int kStageBytes = kOperandBytes + W / 2 * kBlockK * 2;  // half the columns' operand in each CTA
  static constexpr int kStages = kRingBytes / kStageBytes;
  static constexpr int kTmemColumns = 2 * W;
  static constexpr int kChunks = W / 64;  // of 32 columns, in a thread
  static constexpr int kHidden = W / 2;   // columns of g, and of u, in a forward tile
};
constexpr int kMostStages = Wide<128>::kStages;
constexpr int kBarrierBytes = 256;
constexpr int kSmem = kRingBytes + kResultWarps * kStagingBytes + 2 * 2 * kHalf * 4 + kBarrierBytes;
// A pair allocates tensor memory on two SMs, so it can hold one's while it waits
// for the other's, and it holds both while it waits for the kernel before.  No
// other kernel that uses tensor memory can be on those SMs meanwhile: this one
// leaves it less shared memory than its barriers need.
static_assert(kSmem <= 232448 && kSmem > 231 * 1000, "227 KB a CTA");
static_assert((2 * kMostStages + 4) * 8 + 8 <= kBarrierBytes, "barriers and the TMEM address");

// One product in tiles.
struct Product {
  CUtensorMap a[2], b[2];
  int32_t items, tiles_m;  // work items = tiles * splits
  FastDiv tiles, band, last, per_matrix;  // tiles of a split, of a band; rows of tiles in the last band, in a matrix
  int32_t blocks0, blocks, splits, matrices;  // stages of the contraction in the first operand pair, and in all
  int32_t rows, cols;      // of a result matrix
  bool a_mn;               // STORE: A is MN-major
  void* result[2];         // STORE: the matrices
  float* parts;            // STORE of a split product: [splits][matrices][rows][cols]
};

// FWD, AGAIN: one product.  STORE: dx's and then the weights' gradients', or one of them.
struct Ffn {
  Product p[2];
  int32_t long_pairs, ahead;  // see Walk
  FfnOut o;
};

// The order in which a pair takes items: the first product's in turn with the
// other pairs, then the second's.  The first `long_pairs` pairs have one more
// of the first product's; the others make up for it with `ahead` of the second
// product's before all take turns again.
struct Walk {
  int32_t i0, i1, taken, pair, pairs;
  int which, item;
  __device__ __forceinline__ Walk(const Ffn& f) {
    pairs = gridDim.x >> 1, pair = blockIdx.x >> 1;
    i0 = pair, taken = pair < f.long_pairs ? f.ahead : 0;
    i1 = f.ahead * (pairs - f.long_pairs) + (pair < f.long_pairs ? pair + pairs : pair) - f.long_pairs;
  }
  __device__ __forceinline__ bool next(const Ffn& f) {
    which = i0 >= f.p[0].items;
    if (!which) {
      item = i0, i0 += pairs;
      return true;
    }
    if (taken < f.ahead) {
      item = pair - f.long_pairs + taken++ * (pairs - f.long_pairs);
      return true;
    }
    item = i1, i1 += pairs;
    return item < f.p[1].items;
  }
};

__device__ unsigned int g_ffn_wait_failures;  // bounded waits that gave up (read by mp_wait_failures)

struct Tile {
  int32_t m, n, k0, k1, split, of;  // row and column of tiles, stages from k0 to k1, which matrix
};
// Items walk the tiles in bands of kBand rows of tiles, column by column, so
// that those in flight together share operands in L2; all tiles of a split
// first.  (Every role does this for every tile, one thread after another: plain
// divisions, or a band whose height is not a constant, take 300 cycles of a tile
// that has 3,000 where the contraction is short.)
//
// A band has 16 rows of tiles in the forward product and 8 in the gradients'.  A
// wave of 76 tiles that is 8 x 9.5 has the fewest different operand rows; twice
// as high a band reads the weights half as often, which pays where the band's
// rows of x stay in L2 (8192 x 4096 x 14336: 16 rows 1057 us, 8 1083, 32 1131;
// gradients 8 rows 2410 us, 16 2445, 32 2522).
template <int EP>
constexpr int kBand = EP == STORE ? 8 : 16;
template <int BAND>
__device__ __forceinline__ Tile tile_of(const Product& f, uint32_t item) {
  Tile t;
  t.split = 0, t.k0 = 0, t.k1 = f.blocks;
  if (f.splits > 1) {
    t.split = div_by(item, f.tiles);
    item -= t.split * f.tiles.d;
    t.k0 = f.blocks * t.split / f.splits;  // below 2^30
    t.k1 = f.blocks * (t.split + 1) / f.splits;
  }
  const uint32_t band = div_by(item, f.band);
  item -= band * f.band.d;
  const bool whole = (int)(band + 1) * BAND <= f.tiles_m;
  t.n = whole ? item / BAND : div_by(item, f.last);
  t.m = band * BAND + item - t.n * (whole ? BAND : f.last.d);
  t.of = div_by(t.m, f.per_matrix);  // 0 unless two matrices are stored
  t.m -= t.of * f.per_matrix.d;
  return t;
}

// 32 accumulators as 16 pairs.
__device__ __forceinline__ float2 pair_of(const uint32_t (&r)[32], int k) {
  return make_float2(__uint_as_float(r[2 * k]), __uint_as_float(r[2 * k + 1]));
}
__device__ __forceinline__ void set_pair(uint32_t (&r)[32], int k, float2 v) {
  r[2 * k] = __float_as_uint(v.x), r[2 * k + 1] = __float_as_uint(v.y);
}

// One warp's way out: 32 rows of 128 or 64 bytes through its staging buffer,
// so that eight or four lanes store a row's bytes together.  Unit c of 16 bytes
// of row r lies at unit c ^ (r % 8), or c ^ (r / 2 % 4) of the shorter rows,
// which spreads writes and reads over the banks.
struct Way {
  uint32_t stage;
  int lane;
  __device__ __forceinline__ void put128(int c, uint4 v) const {
    sts16(stage + lane * 128 + ((c ^ (lane & 7)) << 4), v.x, v.y, v.z, v.w);
  }
  __device__ __forceinline__ void put64(int c, uint4 v) const {
    sts16(stage + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4), v.x, v.y, v.z, v.w);
  }
  // Rows `pitch` bytes apart from `to`; `rows` of them and `bytes` of each are in the matrix.
  template <int BYTES>
  __device__ __forceinline__ void send(void* to, int64_t pitch, int rows, int bytes) const {
    constexpr int U = BYTES / 16;  // lanes to a row
    __syncwarp();
    const int u = lane % U, r0 = lane / U;
    unsigned char* at = static_cast<unsigned char*>(to) + r0 * pitch + u * 16;
#pragma unroll
    for (int i = 0; i < U; ++i, at += pitch * (32 / U)) {
      const int r = i * (32 / U) + r0, swizzled = U == 8 ? u ^ (r & 7) : u ^ ((r >> 1) & 3);
      const uint4 v = lds16(stage + r * BYTES + (swizzled << 4));
      if (r < rows && u * 16 < bytes) *reinterpret_cast<uint4*>(at) = v;
    }
    __syncwarp();
  }
  // 32 or 64 values of each row, rounded
  template <bool BF16>
  __device__ __forceinline__ void send16(const uint32_t (&r)[32], void* to, int64_t pitch, int rows, int cols) const {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      put64(c, make_uint4(pack16<BF16>(pair_of(r, 4 * c)), pack16<BF16>(pair_of(r, 4 * c + 1)),
                          pack16<BF16>(pair_of(r, 4 * c + 2)), pack16<BF16>(pair_of(r, 4 * c + 3))));
    send<64>(to, pitch * 2, rows, cols * 2);
  }
  template <bool BF16>
  __device__ __forceinline__ void send16(const uint32_t (&lo)[32], const uint32_t (&hi)[32], void* to, int64_t pitch,
                                         int rows, int cols) const {
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const uint32_t(&r)[32] = c < 4 ? lo : hi;
      const int k = (c & 3) * 4;
      put128(c, make_uint4(pack16<BF16>(pair_of(r, k)), pack16<BF16>(pair_of(r, k + 1)), pack16<BF16>(pair_of(r, k + 2)),
                           pack16<BF16>(pair_of(r, k + 3))));
    }
    send<128>(to, pitch * 2, rows, cols * 2);
  }
};

// |values| of 32 columns: NaN-propagating maximum as bits that order as integers.
__device__ __forceinline__ uint32_t amax32(const uint32_t (&r)[32]) {
  float a = 0.0f, b = 0.0f;
#pragma unroll
  for (int k = 0; k < 32; k += 4) {
    a = max3_abs_nan(a, __uint_as_float(r[k]), __uint_as_float(r[k + 1]));
    b = max3_abs_nan(b, __uint_as_float(r[k + 2]), __uint_as_float(r[k + 3]));
  }
  return __float_as_uint(max3_abs_nan(a, b, b));
}

// Codes of 32 columns of this lane's row of 64 bytes, at 16-byte unit `unit`.
__device__ __forceinline__ void codes32(const uint32_t (&r)[32], const Way& way, int unit, uint32_t m, float mul,
                                        bool e5m2, bool mx) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float2 v[kPairs];
#pragma unroll
    for (int k = 0; k < kPairs; ++k) v[k] = pair_of(r, h * kPairs + k);
    uint4 c;
    if (__builtin_expect(m >= kInfBits, 0))
      c = mx ? make_uint4(0u, 0u, 0u, 0u) : nonfinite_unit(v, [&](int i) { return float_sign80(v, i); });
    else
      c = e5m2 ? cast_unit<true>(v, mul) : cast_unit<false>(v, mul);
    way.put64(unit + h, c);
  }
}

// A place in the ring of stages: its number, and the parity of the phase that a
// full stage completes.
template <int STAGES>
struct Turn {
  uint32_t s = 0, parity = 0;
  __device__ __forceinline__ void step() {
    if (++s == STAGES) s = 0, parity ^= 1;
  }
};

// A row's 128 columns are in two threads, `half` 0 and 1: the larger of both;
// NaN for the other thread where this one's sums are not complete (!ok).
__device__ __forceinline__ uint32_t both_halves(uint32_t m, bool ok, uint32_t* slot, int half, int row, int quad) {
  slot[half * kHalf + row] = complete_or_nan(ok, m);
  named_barrier(1 + quad, 64);
  return max(m, slot[(half ^ 1) * kHalf + row]);
}

template <bool BF16, int EP, int W>
__global__ __launch_bounds__(kThreads, 1) void k_ffn(const __grid_constant__ Ffn f) {
  using G = Wide<W>;
  constexpr int kStages = G::kStages, kStageBytes = G::kStageBytes, N = G::kChunks, H = N / 2;
  static_assert(EP != FWD8 || W == 256, "a tile of scales has 128 columns");
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char* const staging = smem + kRingBytes;
  uint32_t* const red = reinterpret_cast<uint32_t*>(staging + kResultWarps * kStagingBytes);  // [2][2][128]
  uint64_t* const full = reinterpret_cast<uint64_t*>(red + 2 * 2 * kHalf);
  uint64_t *const empty = full + kStages, *const tfull = empty + kStages, *const tempty = tfull + 2;
  uint32_t* const tmem_at = reinterpret_cast<uint32_t*>(tempty + 2);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int run = W == 128 ? kLongRun : run_of<EP>(f.o);  // no checkpoint in narrow tiles

  if (warp == kResultWarps && lane == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(full + s, 1), mbar_init(empty + s, 1);
    for (int b = 0; b < 2; ++b) mbar_init(tfull + b, 1), mbar_init(tempty + b, 2 * kResultWarps);
    fence_mbar_init();
  }
  if (warp >= kResultWarps + 2) {  // the maps are on their way meanwhile
    const Product& q = f.p[f.p[0].items == 0];
    const bool of_a = warp & 1;
    if (lane < (of_a ? (EP == STORE ? 2 : 1) : (EP == STORE && q.a_mn ? 1 : 2))) prefetch_tensor_map((of_a ? q.a : q.b) + lane);
  }
  if (warp == kResultWarps + 1) tmem_alloc<2>(smem_u32(tmem_at), G::kTmemColumns);
  tmem_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers stand
  tmem_fence_after();
  const uint32_t tmem = *tmem_at;
  chain_wait();
  chain_release();

  bool ok = true;
  if (warp >= kResultWarps) {
    fewer_registers<kOtherRegisters>();
    if ((warp == kResultWarps || warp == kResultWarps + 2) && lane == 0) {
      // Operand tiles: one warp copies A's, another B's.  (One for both issued
      // up to four copies a stage and held the MN-major products back: the
      // weights' gradients of 8192 x 4096 x 14336 took 1280 us, then 1125.)
      const bool is_b = warp != kResultWarps;
      const uint32_t bars = map_rank(smem_u32(full), 0), tiles = smem_u32(smem) + (is_b ? kOperandBytes : 0);
      Turn<kStages> at_stage;
      uint32_t filled = 0;  // stages that have been filled, kStages at most
      for (Walk w(f); ok && w.next(f);) {
        const Product& q = f.p[w.which];
        const Tile t = tile_of<kBand<EP>>(q, w.item);
        const bool mn = EP == STORE && (is_b || q.a_mn);
        int at;                             // the first of the tile's 128 rows of this operand in this CTA
        const CUtensorMap *map0, *map1;     // of the first operand pair and of the second
        if (!is_b) {
          at = t.m * 2 * kHalf + rank * kHalf;
          map0 = q.a + t.of, map1 = q.a + 1;
        } else if (EP == STORE) {
          at = t.n * W + rank * (W / 2);
          map0 = q.b, map1 = q.b + 1;
        } else {
          at = t.n * G::kHidden;
          map0 = map1 = q.b + rank;
        }
        for (int kb = t.k0; kb < t.k1; ++kb, at_stage.step()) {
          const uint32_t s = at_stage.s;
          if (!(ok = mbar_wait_bounded(empty + s, at_stage.parity ^ 1))) break;
          if (filled < kStages) ++filled;
          if (rank == 0 && !is_b) mbar_arrive_expect_tx(full + s, 2 * kStageBytes);
          const uint32_t bar = bars + s * 8, to = tiles + s * kStageBytes;
          const bool second = kb >= q.blocks0;
          const int k = (second ? kb - q.blocks0 : kb) * kBlockK;
          const CUtensorMap* map = second ? map1 : map0;
          if (mn) {
            tma_load_2d_pair(to, map, at, k, bar);
            if (W == 256 || !is_b) tma_load_2d_pair(to + kMnBlockBytes, map, at + 64, k, bar);
          } else {
            tma_load_2d_pair(to, map, k, at, bar);
          }
        }
      }
      // The last arrivals at `empty` come from the other CTA: wait for them.
      if (filled < kStages) at_stage = Turn<kStages>();
      for (uint32_t j = 0; j < filled && ok; ++j, at_stage.step())
        ok = mbar_wait_bounded(empty + at_stage.s, at_stage.parity ^ (filled == kStages));
    } else if (warp == kResultWarps + 1 && lane == 0 && rank == 0) {  // matrix instructions
      Turn<kStages> at_stage;
      uint32_t chunk = 0;
      for (Walk w(f); ok && w.next(f);) {
        const Product& q = f.p[w.which];
        const Tile t = tile_of<kBand<EP>>(q, w.item);
        constexpr bool B_MN = EP == STORE;
        const bool a_mn = B_MN && q.a_mn;
        const uint32_t idesc = a_mn ? instr_desc<BF16, true, B_MN>(2 * kHalf, W)
                                    : instr_desc<BF16, false, B_MN>(2 * kHalf, W);
        const uint32_t step = a_mn ? kDescStep<true> : kDescStep<false>;
        for (int k0 = t.k0; k0 < t.k1 && ok; k0 += run, ++chunk) {
          const uint32_t b = chunk & 1, d = tmem + b * W;
          if (!(ok = mbar_wait_bounded(tempty + b, ((chunk >> 1) & 1) ^ 1))) break;
          tmem_fence_after();
          const int k1 = min(t.k1, k0 + run);
          for (int kb = k0; kb < k1; ++kb, at_stage.step()) {
            const uint32_t s = at_stage.s;
            if (!(ok = mbar_wait_bounded(full + s, at_stage.parity))) break;
            tmem_fence_after();
            const uint32_t pa = smem_u32(smem + s * kStageBytes);
            const uint64_t da = a_mn ? operand_desc<true>(pa) : operand_desc<false>(pa);
            const uint64_t db = operand_desc<B_MN>(pa + kOperandBytes);
#pragma unroll
            for (int j = 0; j < kBlockK / 16; ++j)
              mma_f16<2>(d, da + j * step, db + j * kDescStep<B_MN>, idesc, kb != k0 || j != 0);
            mma_commit<2>(empty + s);
          }
          if (ok) mma_commit<2>(tfull + b);
        }
      }
      if (!ok) for (int s = 0; s < kStages; ++s) mbar_drain(full + s);
    }
  } else {  // results
    more_registers<kResultRegisters>();
    const int quad = warp & 3, half = warp >> 2, in_cta = quad * 32 + lane;
    const Way way{smem_u32(staging + warp * kStagingBytes), lane};
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    uint32_t chunk = 0;
    for (Walk w(f); w.next(f);) {
      const Product& q = f.p[w.which];
      const Tile t = tile_of<kBand<EP>>(q, w.item);
      const int row0 = t.m * 2 * kHalf + rank * kHalf + quad * 32, row = row0 + lane;
      // FWD, AGAIN: acc[j] are 32 columns of g and acc[H + j] the same of u.  STORE: half of the tile's columns.
      uint32_t acc[N][32];
      auto column = [&](int j) {
        return EP == STORE ? half * (W / 2) + j * 32 : j / H * G::kHidden + half * (W / 4) + j % H * 32;
      };
      // Waits for a run's sums; where they are.  After a wait that gave up, the
      // warp goes through its steps (others may wait for it at a barrier)
      // without waiting or storing.
      auto run_done = [&]() {
        ok = ok && __all_sync(0xFFFFFFFFu, mbar_wait_bounded(tfull + (chunk & 1), (chunk >> 1) & 1));
        tmem_fence_after();
        return lanes + (chunk & 1) * W;
      };
      auto run_read = [&]() {  // their place is free
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(map_rank(smem_u32(tempty + (chunk & 1)), 0));
        ++chunk;
      };
      {  // the first run's sums straight to where they stay
        const uint32_t at = run_done();
#pragma unroll
        for (int j = 0; j < N; ++j) tmem_load32(acc[j], at + column(j));
        tmem_wait();
#pragma unroll
        for (int j = 0; j < N; ++j) loaded(acc[j]);
        run_read();
      }
      for (int k0 = t.k0 + run; k0 < t.k1; k0 += run) {
        const uint32_t at = run_done();
        // the next 16 columns on their way while 16 are added
        uint32_t r[2][16];
        tmem_load16(r[0], at + column(0));
#pragma unroll
        for (int j = 0; j < 2 * N; ++j) {
          tmem_wait();
          loaded(r[j & 1]);
          if (j < 2 * N - 1) tmem_load16(r[(j + 1) & 1], at + column((j + 1) >> 1) + ((j + 1) & 1) * 16);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float2 v = make_float2(__uint_as_float(r[j & 1][2 * k]), __uint_as_float(r[j & 1][2 * k + 1]));
            const int to = (j & 1) * 8 + k;
            set_pair(acc[j >> 1], to, add2(pair_of(acc[j >> 1], to), v));
          }
        }
        run_read();
      }
      const int rows = ok ? q.rows : 0;

      if constexpr (EP == STORE) {
        const int col0 = t.n * W + half * (W / 2);
        if (W == 256 && q.splits > 1) {  // narrow tiles are not split
          float* const to = q.parts + ((int64_t)t.split * q.matrices + t.of) * q.rows * q.cols +
                            (int64_t)row0 * q.cols + col0;
#pragma unroll
          for (int j = 0; j < N; ++j) {
#pragma unroll
            for (int c = 0; c < 8; ++c)
              way.put128(c, make_uint4(acc[j][4 * c], acc[j][4 * c + 1], acc[j][4 * c + 2], acc[j][4 * c + 3]));
            way.send<128>(to + j * 32, (int64_t)q.cols * 4, rows - row0, (q.cols - col0 - j * 32) * 4);
          }
        } else {
          uint16_t* const to = static_cast<uint16_t*>(q.result[t.of]) + (int64_t)row0 * q.cols + col0;
#pragma unroll
          for (int j = 0; j < H; ++j)
            way.send16<BF16>(acc[2 * j], acc[2 * j + 1], to + j * 64, q.cols, rows - row0, q.cols - col0 - j * 64);
        }
      } else {
        const int col0 = t.n * G::kHidden + half * (W / 4);
        const int down = rows - row0, across = q.cols - col0;  // what is left of the matrix
        const int64_t at = (int64_t)row0 * q.cols + col0;
        // 32 H rounded columns from acc[first] on
        auto send = [&](auto first, void* base, int64_t from, int64_t pitch) {
          constexpr int k = decltype(first)::value;
          uint16_t* const to = static_cast<uint16_t*>(base) + from;
          if constexpr (H == 2)
            way.send16<BF16>(acc[k], acc[k + 1], to, pitch, down, across);
          else
            way.send16<BF16>(acc[k], to, pitch, down, across);
        };
        constexpr auto of_g = std::integral_constant<int, 0>{};
        constexpr auto of_u = std::integral_constant<int, H>{};
        if (col0 + W / 4 > q.cols) {  // columns past the end: 0 * inf has made NaN of them in a row with infinities
#pragma unroll
          for (int j = 0; j < N; ++j)
#pragma unroll
            for (int k = 0; k < 32; ++k) acc[j][k] = col0 + j % H * 32 + k < q.cols ? acc[j][k] : 0u;
        }
        if constexpr (EP == AGAIN) {
          const uint4* from = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(f.o.dp) +
                                                              ((int64_t)row * q.cols + col0));
#pragma unroll
          for (int c = 0; c < 4 * H; ++c) {
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (row < rows && col0 + c * 8 < q.cols) v = ld_plain(from + c);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int j = c >> 2, k = (c & 3) * 4 + i;
              float2 dg, du;
              slopes(pair16<BF16>(w[i]), pair_of(acc[j], k), pair_of(acc[H + j], k), &dg, &du);
              set_pair(acc[j], k, dg);
              set_pair(acc[H + j], k, du);
            }
          }
          send(of_g, f.o.dg, at, q.cols);
          send(of_u, f.o.du, at, q.cols);
        } else {
          const int tile = t.n;  // 128 columns are a tile of scales
          if (f.o.gate) {
            const int64_t kept = (int64_t)row0 * f.o.ld + col0;
            send(of_g, f.o.gate, kept, f.o.ld);
            send(of_u, f.o.up, kept, f.o.ld);
          }
          if constexpr (W == 256)  // a tile of scales has 128 columns
            if (f.o.ckpt) {
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const uint32_t m = both_halves(max(amax32(acc[2 * j]), amax32(acc[2 * j + 1])), ok, red + j * 2 * kHalf,
                                               half, in_cta, quad);
                float mul;
                const float scale = tile_scale(m, 448.0f, &mul);
                if (half == 0 && row < rows) f.o.ckpt_scales[((int64_t)j * q.rows + row) * f.o.tiles + tile] = scale;
                codes32(acc[2 * j], way, 0, m, mul, false, false);
                codes32(acc[2 * j + 1], way, 2, m, mul, false, false);
                way.send<64>(f.o.ckpt + (int64_t)j * q.rows * q.cols + at, q.cols, down, across);
              }
              named_barrier(1 + quad, 64);  // the slots have been read
            }
#pragma unroll
          for (int j = 0; j < H; ++j)
#pragma unroll
            for (int k = 0; k < 16; ++k) set_pair(acc[j], k, gated(pair_of(acc[j], k), pair_of(acc[H + j], k)));
          if constexpr (EP == FWD16) {
            send(of_g, f.o.p, at, q.cols);
          } else {
            uint32_t m[2] = {amax32(acc[0]), amax32(acc[1])};
            float mul[2];
            if (f.o.mx) {
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                uint32_t byte;
                mx_scale(m[j], f.o.e5m2 ? 15u : 8u, &mul[j], &byte);
                if (row < rows && col0 + j * 32 < q.cols)
                  static_cast<uint8_t*>(f.o.p_scales)[(int64_t)row * f.o.per_row + (col0 >> 5) + j] = (uint8_t)byte;
              }
            } else {
              m[0] = m[1] = both_halves(max(m[0], m[1]), ok, red, half, in_cta, quad);
              const float scale = tile_scale(m[0], f.o.e5m2 ? 57344.0f : 448.0f, &mul[0]);
              mul[1] = mul[0];
              if (half == 0 && row < rows) static_cast<float*>(f.o.p_scales)[(int64_t)row * f.o.per_row + tile] = scale;
              named_barrier(1 + quad, 64);  // the slot has been read
            }
            codes32(acc[0], way, 0, m[0], mul[0], f.o.e5m2, f.o.mx);
            codes32(acc[1], way, 2, m[1], mul[1], f.o.e5m2, f.o.mx);
            way.send<64>(static_cast<uint8_t*>(f.o.p) + at, q.cols, down, across);
          }
        }
      }
    }
  }
  if (!ok) atomicAdd(&g_ffn_wait_failures, 1u);
  tmem_fence_before();
  __syncthreads();
  cluster_sync();  // no CTA leaves while the other's instructions may read or signal it
  tmem_fence_after();
  if (warp == kResultWarps + 1) tmem_free<2>(tmem, G::kTmemColumns);
}

// Adds the parts of up to two products split along their contraction, in order,
// and rounds once.  One thread: 8 elements.
struct Join {
  const float* parts[2];
  int32_t splits[2];
  int64_t n[2], one[2];  // elements of all matrices of a product, and of one
  void* out[2][2];
  unsigned first;        // CTAs of the first
};
template <bool BF16>
__global__ __launch_bounds__(256) void k_ffn_join(const __grid_constant__ Join f) {
  chain_wait();
  chain_release();
  const int w = blockIdx.x >= f.first;
  const int64_t i = ((int64_t)(blockIdx.x - (w ? f.first : 0)) * 256 + threadIdx.x) * 8, n = f.n[w], one = f.one[w];
  if (i >= n) return;
  float2 v[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = make_float2(0.0f, 0.0f);
#pragma unroll 4
  for (int s = 0; s < f.splits[w]; ++s) {
    const float4* p = reinterpret_cast<const float4*>(f.parts[w] + s * n + i);
    const float4 a = __ldcg(p), b = __ldcg(p + 1);
    v[0] = add2(v[0], make_float2(a.x, a.y)), v[1] = add2(v[1], make_float2(a.z, a.w));
    v[2] = add2(v[2], make_float2(b.x, b.y)), v[3] = add2(v[3], make_float2(b.z, b.w));
  }
  uint16_t* to = i < one ? static_cast<uint16_t*>(f.out[w][0]) + i : static_cast<uint16_t*>(f.out[w][1]) + (i - one);
  *reinterpret_cast<uint4*>(to) = make_uint4(pack16<BF16>(v[0]), pack16<BF16>(v[1]), pack16<BF16>(v[2]), pack16<BF16>(v[3]));
}

// Pairs of CTAs that the device runs at once.
int64_t most_pairs() { return sm_count() < 2 ? 1 : sm_count() / 2; }

// Evens out what the pairs have to do (Walk) with `a` items of the first product
// and `b` of the second: those without the last turn's item of the first take as
// many stages of the second ahead.  (A tile of a short contraction takes six
// stages' time, for its results' way out.)
struct Turns {
  int long_pairs, ahead;
};
Turns turns_of(int64_t a, int64_t a_stages, int64_t b, int64_t b_stages, int64_t pairs) {
  Turns t{(int)(a % pairs), 0};
  if (t.long_pairs == 0 || b == 0) return t;
  const int64_t one = b_stages > 6 ? b_stages : 6, longer = ((a_stages > 6 ? a_stages : 6) + one / 2) / one;
  const int64_t others = pairs - t.long_pairs;
  t.ahead = (int)(longer < b / others ? longer : b / others);
  return t;
}
// When the last pair is done, in stages of 256 columns, results' way out included.
int64_t end_of(int64_t a, int64_t a_stages, int64_t a_out, int64_t b, int64_t b_stages, int64_t b_out) {
  const int64_t pairs = a + b < most_pairs() ? a + b : most_pairs();
  const Turns t = turns_of(a, a_stages, b, b_stages, pairs);
  const int64_t rest = (b - t.ahead * (pairs - t.long_pairs) + pairs - 1) / pairs, each = a / pairs;
  const int64_t ca = a_stages + a_out, cb = b_stages + b_out;
  const int64_t longs = t.long_pairs ? (each + 1) * ca + rest * cb : 0, others = each * ca + (t.ahead + rest) * cb;
  return longs > others ? longs : others;
}
// Stages of 256 columns that stages of 128 take: half the matrix instructions, but
// three quarters of the operands, and their copies bound them.
int64_t narrow_stages(int64_t blocks) { return (blocks * 7 + 7) / 8; }

template <bool BF16, int EP, int W>
mp_status launch(Ffn& f, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  const auto kernel = k_ffn<BF16, EP, W>;
  if (!smem_opt_in(kernel, kSmem, done)) return MP_ECUDA;
  const Product &a = f.p[0], &b = f.p[1];
  const int64_t items = (int64_t)a.items + b.items;
  const int pairs = (int)(items < most_pairs() ? items : most_pairs());
  const Turns t = turns_of(a.items, a.items ? a.blocks / a.splits : 0, b.items, b.items ? b.blocks / b.splits : 0, pairs);
  f.long_pairs = t.long_pairs, f.ahead = t.ahead;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2, attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * pairs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
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

bool type16(mp_dtype t) { return t == MP_F16 || t == MP_BF16; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
// Tiles, and the walk over them.
void lay_out(Product& f, int matrices, int rows_of_tiles, int tiles_n, int splits, int band) {
  f.matrices = matrices, f.splits = splits;
  f.tiles_m = matrices * rows_of_tiles;
  f.items = f.tiles_m * tiles_n * splits;
  f.tiles = fast_div(f.tiles_m * tiles_n), f.band = fast_div(band * tiles_n);
  f.last = fast_div(f.tiles_m % band ? f.tiles_m % band : band), f.per_matrix = fast_div(rows_of_tiles);
}

// The gradients' products: tiles and stages of the contraction of dx (none up to
// kFewDxRows rows, which have a kernel of their own) and of the weights' gradients,
// and into how many parts each is split along its contraction.  With all pairs
// at work on both products each would have `even` stages to do; a tile longer
// than that by a quarter or more is split into parts of at most about that length,
// of four stages at least, if that saves 16 stages, what the parts' way through
// memory costs.  Or both products have whole tiles of 128 columns, where that
// ends a sixth earlier by what the steps have measured: a tile's results take 6
// stages' time on their way out, 3 with 128 columns, 11 in parts, and the launch
// that joins them 24 (2048 x 256 x 688 11.5 us, in tiles of 256, split, 16.1; 1024 x
// 1024 x 256 7.5 and 8.6; 301 x 1040 x 1456 18.3 and 15.8; 260 x 768 x 2992 28.8 and
// 18.8).  Whichever gradients are asked for, the tiles and parts are these, so
// that results do not depend on that.
struct Plan {
  int64_t dx_tiles, dw_tiles;
  int dx_blocks, dw_blocks, dx_splits, dw_splits;
  bool narrow;                // tiles of 128 columns
  size_t dx_parts, dw_parts;  // bytes
};
int splits_of(int64_t tiles, int blocks, int64_t even) {
  int64_t s = blocks / even;
  if (s == 1 && blocks > even + even / 4) s = 2;
  if (s > blocks / 4) s = blocks / 4;
  return s < 2 || tiles == 0 || blocks - blocks / s < 16 ? 1 : s < 16 ? (int)s : 16;
}
Plan plan_of(int64_t rows, int64_t width, int64_t hidden) {
  Plan p;
  p.dx_blocks = 2 * ceil_div(hidden, kBlockK), p.dw_blocks = ceil_div(rows, kBlockK);
  const auto tiles = [&](int columns) {
    p.dx_tiles = rows <= kFewDxRows ? 0 : (int64_t)ceil_div(rows, 2 * kHalf) * ceil_div(width, columns);
    p.dw_tiles = 2ll * ceil_div(hidden, 2 * kHalf) * ceil_div(width, columns);
  };
  tiles(128);
  const int64_t narrow = end_of(p.dx_tiles, narrow_stages(p.dx_blocks), 3, p.dw_tiles, narrow_stages(p.dw_blocks), 3);
  tiles(256);
  const auto least = [](int blocks) { return blocks > 6 ? blocks : 6; };
  const int64_t even =
      (p.dx_tiles * least(p.dx_blocks) + p.dw_tiles * least(p.dw_blocks) + most_pairs() - 1) / most_pairs();
  p.dx_splits = splits_of(p.dx_tiles, p.dx_blocks, even), p.dw_splits = splits_of(p.dw_tiles, p.dw_blocks, even);
  const int64_t wide = end_of(p.dx_tiles * p.dx_splits, p.dx_blocks / p.dx_splits, p.dx_splits > 1 ? 11 : 6,
                              p.dw_tiles * p.dw_splits, p.dw_blocks / p.dw_splits, p.dw_splits > 1 ? 11 : 6) +
                       (p.dx_splits > 1 || p.dw_splits > 1 ? 24 : 0);
  p.narrow = narrow * 6 < wide * 5;
  if (p.narrow) {
    tiles(128);
    p.dx_splits = p.dw_splits = 1;
  }
  p.dx_parts = p.dx_splits > 1 ? (size_t)p.dx_splits * rows * width * 4 : 0;
  p.dw_parts = p.dw_splits > 1 ? (size_t)p.dw_splits * 2 * hidden * width * 4 : 0;
  return p;
}

// The products of f, and the joining of those that are split.
mp_status multiply(bool bf16, bool narrow, Ffn& f, cudaStream_t st) {
  const mp_status s = bf16 ? narrow ? launch<true, STORE, 128>(f, st) : launch<true, STORE, 256>(f, st)
                           : narrow ? launch<false, STORE, 128>(f, st) : launch<false, STORE, 256>(f, st);
  if (s != MP_OK) return s;
  Join j = {};
  unsigned ctas[2] = {0, 0};
  for (int w = 0; w < 2; ++w) {
    const Product& q = f.p[w];
    if (q.items == 0 || q.splits == 1) continue;
    j.parts[w] = q.parts, j.splits[w] = q.splits;
    j.one[w] = (int64_t)q.rows * q.cols, j.n[w] = q.matrices * j.one[w];
    j.out[w][0] = q.result[0], j.out[w][1] = q.result[1];
    ctas[w] = (unsigned)((j.n[w] / 8 + 255) / 256);
  }
  if (ctas[0] + ctas[1] == 0) return MP_OK;
  j.first = ctas[0];
  launch_chained(bf16 ? k_ffn_join<true> : k_ffn_join<false>, dim3(ctas[0] + ctas[1]), dim3(256), 0, st, j);
  note_launches(1);
  return launch_status();
}

// Rows, columns and row lengths that both calls take.
bool shape_ok(int64_t rows, int64_t width, int64_t hidden, int step) {
  if (rows >= (1ll << 31) - 256 || width > (1 << 20) || hidden > (1 << 20)) return false;
  if (width % 16 != 0 || hidden % step != 0) return false;
  return ceil_div(rows, 256) * (int64_t)ceil_div(2 * hidden + width, 128) < (1ll << 30);
}
bool pitch_ok(int64_t ld, int64_t cols, int64_t rows) {
  return rows <= 1 || (ld >= cols && ld < (1ll << 61) / rows && ld % 8 == 0);
}

// Whether tiles of 128 columns end earlier: a wave takes its stages, or the ten (or
// five) that a tile's activation and results take, which the last wave adds (301 x
// 1040 x 1456 7.5 us, in tiles of 256 9.5; 1000 x 1024 x 1024 7.7 and 9.3; 260 x 768 x
// 2992 9.3 and 8.1; 700 x 4096 x 4096 46 and 40.5).
bool narrow_forward(int64_t tiles_m, int64_t hidden, int blocks) {
  const auto end = [&](int columns, int64_t stages, int64_t out) {
    const int64_t waves = (tiles_m * ceil_div(hidden, columns) + most_pairs() - 1) / most_pairs();
    return waves * (stages > out ? stages : out) + out;
  };
  return end(Wide<128>::kHidden, narrow_stages(blocks), 5) < end(Wide<256>::kHidden, blocks, 10);
}

// Forms g and u (FWD16, FWD8, AGAIN).
template <int EP>
mp_status project(bool bf16, const void* x, const void* w_gate, const void* w_up, int64_t rows, int64_t width,
                  int64_t hidden, const FfnOut& o, cudaStream_t st) {
  if (few_forward(rows, width, hidden)) return ffn_few_project(EP, bf16, x, w_gate, w_up, rows, width, hidden, o, st);
  Ffn f = {};
  Product& q = f.p[0];
  q.blocks = q.blocks0 = ceil_div(width, kBlockK);
  const bool narrow = EP != FWD8 && !o.ckpt && narrow_forward(ceil_div(rows, 2 * kHalf), hidden, q.blocks);
  const int box = narrow ? Wide<128>::kHidden : Wide<256>::kHidden;
  if (!map16(&q.a[0], x, rows, width, width, kHalf) || !map16(&q.b[0], w_gate, hidden, width, width, box) ||
      !map16(&q.b[1], w_up, hidden, width, width, box))
    return MP_ECUDA;
  f.o = o;
  q.rows = (int32_t)rows, q.cols = (int32_t)hidden;
  lay_out(q, 1, ceil_div(rows, 2 * kHalf), ceil_div(hidden, box), 1, kBand<EP>);
  if constexpr (EP != FWD8) {
    if (narrow) return bf16 ? launch<true, EP, 128>(f, st) : launch<false, EP, 128>(f, st);
  }
  return bf16 ? launch<true, EP, 256>(f, st) : launch<false, EP, 256>(f, st);
}

}  // namespace

uint32_t ffn_wait_failures() {  // of both kernels
  uint32_t v = 0;
  if (cudaMemcpyFromSymbol(&v, g_ffn_wait_failures, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
  const uint32_t w = ffn_few_wait_failures();
  return v > UINT32_MAX - w ? UINT32_MAX : v + w;
}

}  // namespace mp

extern "C" MP_API mp_status linear_swiglu(const void* x, mp_dtype x_dtype, int64_t rows, int64_t width, int64_t hidden,
                                          const void* w_gate, const void* w_up, void* p, mp_dtype p_dtype,
                                          int32_t scale_block, void* p_scales, void* gate, void* up, int64_t ld,
                                          void* ckpt, float* ckpt_scales, void* stream) {
  using namespace mp;
  if (rows < 0 || width < 0 || hidden < 0 || !type16(x_dtype)) return MP_EINVAL;
  const bool fp8 = p_dtype == MP_E4M3 || p_dtype == MP_E5M2;
  if (!fp8 && p_dtype != x_dtype) return MP_EINVAL;
  if (fp8 && scale_block != 128 && scale_block != 32) return MP_EINVAL;
  if (!shape_ok(rows, width, hidden, fp8 && scale_block == 32 ? 32 : 16)) return MP_ESHAPE;
  if (rows == 0 || hidden == 0) return MP_OK;
  if (width == 0) return MP_ESHAPE;
  if (!x || !w_gate || !w_up || !p || fp8 != (p_scales != nullptr) || (!gate != !up) || (!ckpt != !ckpt_scales) ||
      (gate && ckpt))
    return MP_EINVAL;
  if (gate && !pitch_ok(ld, hidden, rows)) return MP_ESHAPE;
  if (!aligned16(x) || !aligned16(w_gate) || !aligned16(w_up) || !aligned16(p) || !aligned16(gate) || !aligned16(up) ||
      !aligned16(ckpt) || !aligned4(ckpt_scales) || (fp8 && scale_block == 128 && !aligned4(p_scales)))
    return MP_EALIGN;
  FfnOut o = {};
  o.p = p, o.p_scales = p_scales, o.e5m2 = p_dtype == MP_E5M2, o.mx = scale_block == 32;
  o.tiles = ceil_div(hidden, 128);
  o.per_row = o.mx ? (int32_t)(hidden / 32) : o.tiles;
  o.gate = gate, o.up = up, o.ld = rows > 1 ? ld : hidden;
  o.ckpt = static_cast<uint8_t*>(ckpt), o.ckpt_scales = ckpt_scales;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf16 = x_dtype == MP_BF16;
  return fp8 ? project<FWD8>(bf16, x, w_gate, w_up, rows, width, hidden, o, st)
             : project<FWD16>(bf16, x, w_gate, w_up, rows, width, hidden, o, st);
}

namespace mp {
namespace {

// The workspace: dg and du [2][rows][hidden] in 16 bits, then the parts of split products.
size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace
}  // namespace mp

extern "C" MP_API size_t linear_swiglu_workspace_size(int64_t rows, int64_t width, int64_t hidden) {
  using namespace mp;
  if (rows <= 0 || width <= 0 || hidden <= 0 || !shape_ok(rows, width, hidden, 16)) return 0;
  const Plan p = plan_of(rows, width, hidden);
  return up256((size_t)rows * hidden * 4) + up256(p.dx_parts) + p.dw_parts;
}

extern "C" MP_API mp_status linear_swiglu_backward(const void* dp, mp_dtype x_dtype, int64_t rows, int64_t width,
                                                   int64_t hidden, const void* x, const void* w_gate, const void* w_up,
                                                   const void* gate, const void* up, int64_t ld, const void* ckpt,
                                                   const float* ckpt_scales, void* dx, void* dw_gate, void* dw_up,
                                                   void* d_workspace, size_t workspace_bytes, void* stream) {
  using namespace mp;
  if (rows < 0 || width < 0 || hidden < 0 || !type16(x_dtype)) return MP_EINVAL;
  if (!shape_ok(rows, width, hidden, 16)) return MP_ESHAPE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (width == 0) return rows == 0 || hidden == 0 ? MP_OK : MP_ESHAPE;
  if ((!dw_gate != !dw_up) || (!gate != !up) || (!ckpt != !ckpt_scales) || (gate && ckpt)) return MP_EINVAL;
  if (!aligned16(dx) || !aligned16(dw_gate) || !aligned16(dw_up)) return MP_EALIGN;
  if (rows == 0 || hidden == 0) {  // empty sums
    if (rows > 0 && dx && cudaMemsetAsync(dx, 0, (size_t)rows * width * 2, st) != cudaSuccess) return MP_ECUDA;
    const size_t n = (size_t)hidden * width * 2;
    if (n && dw_gate && (cudaMemsetAsync(dw_gate, 0, n, st) != cudaSuccess || cudaMemsetAsync(dw_up, 0, n, st) != cudaSuccess))
      return MP_ECUDA;
    return MP_OK;
  }
  if (!dx && !dw_gate) return MP_OK;
  if (!dp || !w_gate || !w_up || !x) return MP_EINVAL;
  if (gate && !pitch_ok(ld, hidden, rows)) return MP_ESHAPE;
  if (!aligned16(dp) || !aligned16(x) || !aligned16(w_gate) || !aligned16(w_up) || !aligned16(gate) || !aligned16(up) ||
      !aligned16(ckpt) || !aligned4(ckpt_scales) || !aligned16(d_workspace))
    return MP_EALIGN;
  if (!d_workspace || workspace_bytes < linear_swiglu_workspace_size(rows, width, hidden)) return MP_EWORKSPACE;
  uint16_t* const dg = static_cast<uint16_t*>(d_workspace);
  uint16_t* const du = dg + rows * hidden;
  unsigned char* const parts = static_cast<unsigned char*>(d_workspace) + up256((size_t)rows * hidden * 4);
  const bool bf16 = x_dtype == MP_BF16;
  if (gate || ckpt) {
    const mp_status s = swiglu_backward(dp, x_dtype, rows, hidden, gate, up, ld, ckpt, ckpt_scales, dg, du, hidden, stream);
    if (s != MP_OK) return s;
  } else {
    FfnOut o = {};
    o.dp = dp, o.dg = dg, o.du = du;
    const mp_status s = project<AGAIN>(bf16, x, w_gate, w_up, rows, width, hidden, o, st);
    if (s != MP_OK) return s;
  }
  if (dx && rows <= kFewDxRows) {
    const mp_status s = ffn_few_dx(bf16, dg, du, w_gate, w_up, rows, width, hidden, dx, st);
    if (s != MP_OK || !dw_gate) return s;
  }
  const Plan plan = plan_of(rows, width, hidden);
  Ffn f = {};
  if (dx && rows > kFewDxRows) {
    Product& q = f.p[0];
    if (!map16(&q.a[0], dg, rows, hidden, hidden, kHalf) || !map16(&q.a[1], du, rows, hidden, hidden, kHalf) ||
        !map16(&q.b[0], w_gate, hidden, width, width, 64) || !map16(&q.b[1], w_up, hidden, width, width, 64))
      return MP_ECUDA;
    q.blocks0 = plan.dx_blocks / 2, q.blocks = plan.dx_blocks;
    q.rows = (int32_t)rows, q.cols = (int32_t)width;
    q.result[0] = dx, q.parts = reinterpret_cast<float*>(parts);
    lay_out(q, 1, ceil_div(rows, 2 * kHalf), ceil_div(width, plan.narrow ? 128 : 256), plan.dx_splits, kBand<STORE>);
  }
  if (dw_gate) {
    Product& q = f.p[1];
    if (!map16(&q.a[0], dg, rows, hidden, hidden, 64) || !map16(&q.a[1], du, rows, hidden, hidden, 64) ||
        !map16(&q.b[0], x, rows, width, width, 64))
      return MP_ECUDA;
    q.blocks0 = q.blocks = plan.dw_blocks, q.a_mn = true;
    q.rows = (int32_t)hidden, q.cols = (int32_t)width;
    q.result[0] = dw_gate, q.result[1] = dw_up, q.parts = reinterpret_cast<float*>(parts + up256(plan.dx_parts));
    lay_out(q, 2, ceil_div(hidden, 2 * kHalf), ceil_div(width, plan.narrow ? 128 : 256), plan.dw_splits, kBand<STORE>);
  }
  return multiply(bf16, plan.narrow, f, st);
}
