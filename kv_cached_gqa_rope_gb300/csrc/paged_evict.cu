// Eviction from a paged cache by accumulated attention weight.
//
// Of a sequence's n > keep cells, each KV head keeps the `recent` last ones
// and, of the others, the keep - recent with the greatest mass (ties: the
// lowest cell).  The kept cells move, in their order, to cells 0 .. keep - 1;
// the pages behind them are free for the scheduler to take.
//
// Kernel 1, one CTA per (sequence, KV head): the (keep - recent)-th greatest
// mass by a radix select over order-preserving 32-bit keys, 11 + 11 + 10 bits
// a pass with a histogram in shared memory, then the list of kept cells in
// ascending order by counting: each warp owns a contiguous stripe, counts its
// kept cells by ballots, and writes them from its prefix on.  The masses are
// read five times, from L2 after the first.
//
// Kernel 2 moves K and V in place: one read and one write of each kept cell
// that moves.  A kept cell's new place is never behind its old one, so in
// ascending order the cells that a batch overwrites were sources of this batch
// or earlier ones: a CTA walks one (sequence, head, K or V, column slice) in
// batches, reads a batch ahead, and a barrier between a batch's reads and its
// writes is all the order that moving in place needs.  Column slices of a row
// do not depend on each other, which is what spreads a few heads over the GPU.
#include <cuda_runtime.h>

#include <algorithm>

#include "paged.cuh"
#include "ptx.cuh"

namespace kvgqa {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;

// Keys in the order of the masses: NaN lowest, then -inf .. +inf, both zeros alike.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (isnan(x)) return 0;
  const uint32_t u = __float_as_uint(x + 0.0f);  // -0 becomes +0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Whether every page of the sequence's n cells is a page of the pool (asked by
// the whole CTA).
__device__ __forceinline__ bool pages_ok(const PagedMeta& m, int a, int n) {
  bool ok = true;
  for (int c = threadIdx.x << m.page_shift; c < n; c += blockDim.x << m.page_shift) ok = ok && paged_page(m, a, c) >= 0;
  return __syncthreads_and(ok);
}

__global__ void __launch_bounds__(kSelThreads) paged_evict_select_kernel(const __grid_constant__ PagedEvictParams p) {
  __shared__ int hist[kBins];
  __shared__ int warp_gt[kSelWarps], warp_eq[kSelWarps];
  __shared__ uint32_t sel_digit;
  __shared__ int sel_need;
  const int a = blockIdx.x / p.H_kv, g = blockIdx.x % p.H_kv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  pdl_trigger();
  const int n = p.m.kv_lengths[a];
  if (n < 0 || n > p.m.max_cells) {
    if (g == 0 && tid == 0) atomicOr(p.status, KVGQA_FLAG_POSITION_RANGE);
    return;
  }
  if (n > p.keep && !pages_ok(p.m, a, n)) {
    if (g == 0 && tid == 0) atomicOr(p.status, KVGQA_FLAG_PAGE_RANGE);
    return;
  }
  const size_t head = static_cast<size_t>(a) * p.H_kv + g;
  const float* mass = p.mass + head * p.mass_cells;
  float* mass_out = p.mass_out + head * p.mass_cells;
  int32_t* kept = p.kept + head * p.keep;
  const int m = min(n, p.keep);
  if (g == 0 && tid == 0) p.new_lengths[a] = m;
  for (int i = m + tid; i < p.mass_cells; i += kSelThreads) mass_out[i] = 0.f;
  for (int i = m + tid; i < p.keep; i += kSelThreads) kept[i] = -1;
  if (n <= p.keep) {
    for (int i = tid; i < n; i += kSelThreads) {
      mass_out[i] = mass[i];
      kept[i] = i;
    }
    return;
  }

  // The smallest key that is kept among the old cells, and how many cells of
  // that very key are.
  const int old = n - p.recent;
  uint32_t thr = 0;       // digits found so far
  int need = p.keep - p.recent;
  if (need > 0) {
    int shift = 32;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int bits = pass == 2 ? 10 : 11;
      const uint32_t above = shift == 32 ? 0u : ~0u << shift;  // digits already fixed
      shift -= bits;
      for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (int i = tid; i < old; i += kSelThreads) {
        const uint32_t k = order_key(mass[i]);
        if ((k & above) == thr) atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1)], 1);
      }
      __syncthreads();
      // From the highest digit down: the first at which the count reaches need.
      // Thread t holds the 4 digits below kBins - 4t.
      int c[4], sum = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) sum += c[i] = hist[kBins - 1 - 4 * tid - i];
      int incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(FULL, incl, o);
        if (lane >= o) incl += t;
      }
      if (lane == 31) warp_gt[warp] = incl;
      __syncthreads();
      int before = incl - sum;
      for (int w = 0; w < warp; ++w) before += warp_gt[w];
      if (before < need && before + sum >= need) {
        int i = 0;
        while (before + c[i] < need) before += c[i++];
        sel_digit = kBins - 1 - 4 * tid - i;
        sel_need = need - before;
      }
      __syncthreads();
      thr |= sel_digit << shift;
      need = sel_need;
    }
  }

  // The kept cells in order.  Stripe of warp w: cells [w * S, w * S + S).
  const int S = ((n + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
  const int s0 = warp * S, s1 = min(n, s0 + S);
  const bool any_old = p.keep > p.recent;
  auto classify = [&](int i, bool& gt, bool& eq, float& x) {
    gt = eq = false;
    x = 0.f;
    if (i < s1) {
      x = mass[i];
      const uint32_t k = order_key(x);
      gt = i >= old || (any_old && k > thr);
      eq = i < old && any_old && k == thr;
    }
  };
  int gts = 0, eqs = 0;
  for (int i = s0 + lane; i < s0 + S; i += 32) {
    bool gt, eq;
    float x;
    classify(i, gt, eq, x);
    gts += __popc(__ballot_sync(FULL, gt));
    eqs += __popc(__ballot_sync(FULL, eq));
  }
  if (lane == 0) {
    warp_gt[warp] = gts;
    warp_eq[warp] = eqs;
  }
  __syncthreads();
  int eq_before = 0, at = 0;  // cells of the threshold's key before this stripe; kept cells before it
  for (int w = 0; w < warp; ++w) {
    at += warp_gt[w];
    eq_before += warp_eq[w];
  }
  at += min(eq_before, need);
  for (int i = s0 + lane; i < s0 + S; i += 32) {
    bool gt, eq;
    float x;
    classify(i, gt, eq, x);
    const uint32_t below = (1u << lane) - 1;
    const uint32_t eqm = __ballot_sync(FULL, eq);
    const bool take = gt || (eq && eq_before + __popc(eqm & below) < need);
    const uint32_t tm = __ballot_sync(FULL, take);
    if (take) {
      const int to = at + __popc(tm & below);
      kept[to] = i;
      mass_out[to] = x;
    }
    at += __popc(tm);
    eq_before += __popc(eqm);
  }
}

constexpr int kMoveThreads = 256;
constexpr int kMoveBatch = 4;  // 16-byte chunks per thread and batch

__global__ void __launch_bounds__(kMoveThreads) paged_evict_move_kernel(const __grid_constant__ PagedEvictParams p,
                                                                        int slices) {
  int b = blockIdx.x;
  const int slice = b % slices;
  b /= slices;
  uint16_t* cache = b & 1 ? p.v_cache : p.k_cache;
  b >>= 1;
  const int a = b / p.H_kv, g = b % p.H_kv;
  pdl_wait();
  const int n = p.m.kv_lengths[a];
  if (n <= p.keep || n > p.m.max_cells || !pages_ok(p.m, a, n)) return;
  const int32_t* kept = p.kept + (static_cast<size_t>(a) * p.H_kv + g) * p.keep;
  const int page = 1 << p.m.page_shift;
  const int chunks = p.D / 8 / slices;  // 16-byte chunks of a row's slice (a power of two)
  const int rows = kMoveThreads / chunks * kMoveBatch;  // rows of a batch
  const int chunk = threadIdx.x % chunks, row = threadIdx.x / chunks;
  auto at = [&](int cell) {
    return cache + ((static_cast<size_t>(paged_page(p.m, a, cell)) * p.H_kv + g) * page + (cell & (page - 1))) * p.D +
           (slice * chunks + chunk) * 8;
  };
  uint4 x[2][kMoveBatch];
  uint16_t* to[2][kMoveBatch];
  auto load = [&](int base, uint4 (&v)[kMoveBatch], uint16_t* (&dst)[kMoveBatch]) {
#pragma unroll
    for (int u = 0; u < kMoveBatch; ++u) {
      const int i = base + row + u * (kMoveThreads / chunks);
      dst[u] = nullptr;
      if (i >= p.keep) continue;
      const int from = kept[i];
      if (from == i) continue;  // already in its place
      dst[u] = at(i);
      v[u] = *reinterpret_cast<const uint4*>(at(from));
    }
  };
  load(0, x[0], to[0]);
  for (int base = 0; base < p.keep; base += 2 * rows) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      load(base + (h + 1) * rows, x[h ^ 1], to[h ^ 1]);
      __syncthreads();  // every read of this batch's cells is done
#pragma unroll
      for (int u = 0; u < kMoveBatch; ++u)
        if (to[h][u]) *reinterpret_cast<uint4*>(to[h][u]) = x[h][u];
    }
  }
}

}  // namespace

cudaError_t launch_paged_evict(const PagedEvictParams& p, cudaStream_t stream) {
  const long long heads = static_cast<long long>(p.m.A) * p.H_kv;
  if (heads == 0) return cudaSuccess;
  // Slices of at least one 32-byte sector, until there are about four CTAs to
  // an SM.
  int slices = 1;
  while (slices < p.D / 16 && heads * 2 * slices < 608) slices *= 2;
  if (heads * 2 * slices > 0x7fffffffll) return cudaErrorInvalidValue;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(heads));
  cfg.blockDim = dim3(kSelThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, paged_evict_select_kernel, p);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(static_cast<unsigned>(heads * 2 * slices));
  cfg.blockDim = dim3(kMoveThreads);
  return cudaLaunchKernelEx(&cfg, paged_evict_move_kernel, p, slices);
}

}  // namespace kvgqa
