// cluster_probe.cu — a test-only kernel for how the parts of a cluster learn of
// a wait that gave up in one of them (failed_part in mp_mma.cuh).  Each of four
// CTAs waits for a barrier on which it arrives itself, but for CTA `silent`,
// whose barrier nothing completes: its wait gives up after the poll limit.  Each
// CTA writes whether it saw a failure.  No memory is touched but the four words.
#include <cstdint>

#include "mp_mma.cuh"

namespace {

constexpr int kParts = 4;

__global__ __cluster_dims__(kParts, 1, 1) void k_cluster_probe(int silent, uint32_t* seen) {
  __shared__ uint64_t bar;
  __shared__ uint32_t failed;
  const int part = (int)mp::cluster_rank(), lane = threadIdx.x;
  bool ok = true;
  if (lane == 0) {
    failed = 0u;
    mp::mbar_init(&bar, 1);
    mp::fence_mbar_init();
    if (part != silent) mp::mbar_arrive(&bar);
    ok = mp::mbar_wait_bounded(&bar, 0);
    if (!ok) failed = 1u;
  }
  __syncwarp();
  mp::cluster_sync();
  const bool any = __any_sync(0xFFFFFFFFu, mp::failed_part(&failed, kParts));
  if (lane == 0) seen[part] = any ? 1u : 0u;
  __syncwarp();
  mp::cluster_sync();
}

}  // namespace

extern "C" int cluster_probe(int silent, uint32_t* d_seen, void* stream) {
  k_cluster_probe<<<kParts, 32, 0, static_cast<cudaStream_t>(stream)>>>(silent, d_seen);
  return cudaGetLastError() == cudaSuccess ? 0 : 1;
}
