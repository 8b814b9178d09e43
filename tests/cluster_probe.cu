// cluster_probe.cu — a test-only kernel for how the parts of a cluster's sum learn
// of a wait that gave up in one of them (complete_or_nan in mp_mma.cuh).  Each of
// four CTAs waits for a barrier on which it arrives itself, but for CTA `silent`,
// whose barrier nothing completes: its wait gives up after the poll limit.  Then
// each adds all four parts, part + 1, in order.  No memory is touched but the four sums.
#include <cstdint>

#include "mp_mma.cuh"

namespace {

constexpr int kParts = 4;

__global__ __cluster_dims__(kParts, 1, 1) void k_cluster_probe(int silent, float* sums) {
  __shared__ uint64_t bar;
  __shared__ __align__(16) float mine[4];
  const int part = (int)mp::cluster_rank(), lane = threadIdx.x;
  if (lane == 0) {
    mp::mbar_init(&bar, 1);
    mp::fence_mbar_init();
    if (part != silent) mp::mbar_arrive(&bar);
    const bool ok = mp::mbar_wait_bounded(&bar, 0);
    for (int i = 0; i < 4; ++i) mine[i] = __uint_as_float(mp::complete_or_nan(ok, __float_as_uint(part + 1.0f)));
  }
  __syncwarp();
  mp::cluster_sync();
  float s = 0.0f;
  for (int p = 0; p < kParts; ++p) s += mp::ld_cluster(mp::map_rank(mp::smem_u32(mine), p)).w;
  if (lane == 0) sums[part] = s;
  __syncwarp();
  mp::cluster_sync();
}

}  // namespace

extern "C" int cluster_probe(int silent, float* d_sums, void* stream) {
  k_cluster_probe<<<kParts, 32, 0, static_cast<cudaStream_t>(stream)>>>(silent, d_sums);
  return cudaGetLastError() == cudaSuccess ? 0 : 1;
}
