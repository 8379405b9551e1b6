// Pages of a paged cache's pools copied to other pages: page src[i] of every pool
// to page dst[i].
//
// Nothing but a copy: bound by memory, and by a launch and a round trip where it is
// short.  A warp copies 4 KB of one page of one pool, 8 loads of 16 bytes a
// lane in flight before the first store; the warp of a page's first 4 KB takes the
// page's scales along.  8192 pages of 32 cells (8 KV heads of 128, codes; 1.07 GB moved)
// take 161 us, 6.67 TB/s, 98 % of a copy's rate; 507 of 4 heads of 64 in FP16 5.8-6.1 us, 80-84 %;
// 16 pages 2.0 us in a graph, 4.1 in calls.
#include <cuda_runtime.h>

#include "kvgqa.h"
#include "kvgqa_internal.h"
#include "ptx.cuh"

namespace kvgqa {
namespace {

constexpr int kWarps = 4;
constexpr int kLoads = 8;                     // 16-byte loads of a lane in flight
constexpr int kSlice = 32 * 16 * kLoads;      // bytes of a warp

__global__ void __launch_bounds__(kWarps * 32) paged_copy_kernel(const __grid_constant__ PagedCopyParams p, int slices) {
  const int lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  const long long unit = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const long long pair = unit / (2 * slices);
  if (pair >= p.n) return;
  const int rest = static_cast<int>(unit - pair * (2 * slices)), which = rest / slices, slice = rest % slices;
  const int src = p.src[pair], dst = p.dst[pair];
  if (src < 0 || src >= p.P || dst < 0 || dst >= p.P) {
    if (lane == 0) atomicOr(p.status, KVGQA_FLAG_PAGE_RANGE);
    return;
  }
  if (src == dst) return;
  const int64_t bytes = p.page_bytes[which];
  const int64_t from = static_cast<int64_t>(slice) * kSlice + lane * 16;
  const unsigned char* s = p.pool[which] + src * bytes;
  unsigned char* d = p.pool[which] + dst * bytes;
  uint4 x[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i)
    if (from + i * 512 < bytes) x[i] = __ldcs(reinterpret_cast<const uint4*>(s + from + i * 512));
#pragma unroll
  for (int i = 0; i < kLoads; ++i)
    if (from + i * 512 < bytes) *reinterpret_cast<uint4*>(d + from + i * 512) = x[i];
  if (slice == 0 && p.pool[2 + which]) {
    const int64_t sb = p.page_bytes[2 + which];
    const unsigned char* ss = p.pool[2 + which] + src * sb;
    unsigned char* sd = p.pool[2 + which] + dst * sb;
    if ((reinterpret_cast<uintptr_t>(p.pool[2 + which]) | sb) % 4 == 0) {
      for (int64_t i = lane * 4; i < sb; i += 128) *reinterpret_cast<uint32_t*>(sd + i) = *reinterpret_cast<const uint32_t*>(ss + i);
    } else {
      for (int64_t i = lane; i < sb; i += 32) sd[i] = ss[i];
    }
  }
}

}  // namespace

cudaError_t launch_paged_copy(const PagedCopyParams& p, cudaStream_t stream) {
  if (p.n == 0 || p.page_bytes[0] == 0) return cudaSuccess;
  const int64_t slices = (p.page_bytes[0] + kSlice - 1) / kSlice;
  const int64_t ctas = (static_cast<int64_t>(p.n) * 2 * slices + kWarps - 1) / kWarps;
  if (slices > 0x3fffffff || ctas > 0x7fffffff) return cudaErrorInvalidValue;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_copy_kernel, p, static_cast<int>(slices));
}

}  // namespace kvgqa
