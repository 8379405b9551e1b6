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
// kept cells by ballots, and writes them from its prefix on.  The masses of up to
// kCachedCells cells are read once and kept in shared memory; those of longer
// sequences are read five times, from L2 after the first.  Each sequence's own
// length decides, however wide the caller's mass is (32 sequences of 1500-8191
// cells in a mass of 65536 a row: 113 us, 119 when the width decided; the zeros
// behind the kept masses are 8 of them).
//
// Kernel 2 moves K and V in place: one read and one write of each kept cell
// that moves.  A kept cell's new place is never behind its old one, so in
// ascending order the cells that a batch overwrites were sources of this batch
// or earlier ones: a CTA walks one (sequence, head, K or V, column slice) in
// batches, reads a batch ahead, and a barrier between a batch's reads and its
// writes is all the order that moving in place needs.  Column slices of a row
// do not depend on each other, which is what spreads a few heads over the GPU.
//
// What bounds it, as measured (8 KV heads of 128): 32 sequences of 1500-8191 cells
// cut to 2048 take 105 us.  The move, 86 of them, runs at 5.7 TB/s read and
// written, 84 % of a copy's rate; the choice is a chain of latencies over a
// head's cells (their load, three counts, two walks), which CTAs of 1024 threads
// shorten from 19 to 17 us.  4 sequences cut to 256 cells take 6.6-6.8 us.
#include <cuda_runtime.h>

#include <algorithm>

#include "paged.cuh"
#include "ptx.cuh"

namespace kvgqa {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
static_assert(kSelWarps <= 32, "a warp adds up the warps' counts");
constexpr int kBins = 2048;
constexpr int kCachedCells = 9216;  // 36 KB of masses beside the histogram: no more than a CTA may have by default

// Keys in the order of the masses: NaN lowest, then -inf .. +inf, both zeros alike.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (isnan(x)) return 0;
  const uint32_t u = __float_as_uint(x + 0.0f);  // -0 becomes +0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

struct SelShared {
  int hist[kBins];
  int warp_gt[kSelWarps], warp_eq[kSelWarps];
  uint32_t digit;
  int need;
};

// The choice of one (sequence a, KV head g) of n cells, by the whole CTA.
// CACHED: the masses of all its cells fit `cells`.
template <bool CACHED>
__device__ __forceinline__ void select_cells(const PagedEvictParams& p, int a, int g, int n, SelShared& sh, float* cells) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const size_t head = static_cast<size_t>(a) * p.H_kv + g;
  const float* mass = p.mass + head * p.mass_cells;
  float* mass_out = p.mass_out + head * p.mass_cells;
  int32_t* kept = p.kept + head * p.keep;
  const int old = n - p.recent;
  if (n > p.keep) {
    // The masses are read once, and the first digits counted, while the table's
    // entries are on their way.
    const int page = tid << p.m.page_shift;
    const int entry = page < n ? paged_page(p.m, a, page) : 0;
    if constexpr (CACHED) {
#pragma unroll 4
      for (int i = tid; i < n; i += kSelThreads) {
        const float x = mass[i];
        cells[i] = x;
        if (i < old) atomicAdd(&sh.hist[order_key(x) >> 21], 1);
      }
    }
    bool ok = entry >= 0;
    for (int c = page + (kSelThreads << p.m.page_shift); c < n; c += kSelThreads << p.m.page_shift)
      ok = ok && paged_page(p.m, a, c) >= 0;
    if (!__syncthreads_and(ok)) {
      if (g == 0 && tid == 0) atomicOr(p.status, KVGQA_FLAG_PAGE_RANGE);
      return;
    }
  }
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

  auto mass_of = [&](int i) {
    if constexpr (CACHED) return cells[i];
    else return mass[i];
  };
  auto key_of = [&](int i) { return order_key(mass_of(i)); };

  // The smallest key that is kept among the old cells, and how many cells of
  // that very key are.
  uint32_t thr = 0;       // digits found so far
  int need = p.keep - p.recent;
  if (need > 0) {
    int shift = 32;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int bits = pass == 2 ? 10 : 11;
      const uint32_t above = shift == 32 ? 0u : ~0u << shift;  // digits already fixed
      shift -= bits;
      if (!CACHED || pass > 0) {
#pragma unroll 4
        for (int i = tid; i < old; i += kSelThreads) {
          const uint32_t k = key_of(i);
          if ((k & above) == thr) atomicAdd(&sh.hist[(k >> shift) & ((1u << bits) - 1)], 1);
        }
        __syncthreads();
      }
      // From the highest digit down: the first at which the count reaches need.
      // Thread t holds the kShare digits below kBins - kShare t.
      constexpr int kShare = kBins / kSelThreads;
      int c[kShare], sum = 0;
#pragma unroll
      for (int i = 0; i < kShare; ++i) {
        sum += c[i] = sh.hist[kBins - 1 - kShare * tid - i];
        sh.hist[kBins - 1 - kShare * tid - i] = 0;  // for the next digits
      }
      int incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(FULL, incl, o);
        if (lane >= o) incl += t;
      }
      if (lane == 31) sh.warp_gt[warp] = incl;
      __syncthreads();
      int before = incl - sum + __reduce_add_sync(FULL, lane < warp ? sh.warp_gt[lane] : 0);
      if (before < need && before + sum >= need) {
        int i = 0;
        while (before + c[i] < need) before += c[i++];
        sh.digit = kBins - 1 - kShare * tid - i;
        sh.need = need - before;
      }
      __syncthreads();
      thr |= sh.digit << shift;
      need = sh.need;
    }
  }

  // The kept cells in order.  Stripe of warp w: cells [w * S, w * S + S).
  const int S = ((n + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
  const int s0 = warp * S, s1 = min(n, s0 + S);
  const bool any_old = p.keep > p.recent;
  auto classify = [&](int i, bool& gt, bool& eq) {
    gt = eq = false;
    if (i < s1) {
      const uint32_t k = key_of(i);
      gt = i >= old || (any_old && k > thr);
      eq = i < old && any_old && k == thr;
    }
  };
  int gts = 0, eqs = 0;
  for (int i = s0 + lane; i < s0 + S; i += 32) {
    bool gt, eq;
    classify(i, gt, eq);
    gts += __popc(__ballot_sync(FULL, gt));
    eqs += __popc(__ballot_sync(FULL, eq));
  }
  if (lane == 0) {
    sh.warp_gt[warp] = gts;
    sh.warp_eq[warp] = eqs;
  }
  __syncthreads();
  // cells of the threshold's key before this stripe; kept cells before it
  int eq_before = __reduce_add_sync(FULL, lane < warp ? sh.warp_eq[lane] : 0);
  int at = __reduce_add_sync(FULL, lane < warp ? sh.warp_gt[lane] : 0) + min(eq_before, need);
  for (int i = s0 + lane; i < s0 + S; i += 32) {
    bool gt, eq;
    classify(i, gt, eq);
    const uint32_t below = (1u << lane) - 1;
    const uint32_t eqm = __ballot_sync(FULL, eq);
    const bool take = gt || (eq && eq_before + __popc(eqm & below) < need);
    const uint32_t tm = __ballot_sync(FULL, take);
    if (take) {
      const int to = at + __popc(tm & below);
      kept[to] = i;
      mass_out[to] = mass_of(i);
    }
    at += __popc(tm);
    eq_before += __popc(eqm);
  }
}

// WIDE: the rows of the mass have room for longer sequences than `cells`.
template <bool WIDE>
__global__ void __launch_bounds__(kSelThreads, 2) paged_evict_select_kernel(const __grid_constant__ PagedEvictParams p) {
  extern __shared__ float cells[];  // of min(mass_cells, kCachedCells) cells
  __shared__ SelShared sh;
  const int a = blockIdx.x / p.H_kv, g = blockIdx.x % p.H_kv;
  pdl_wait();
  pdl_trigger();
  const int n = p.m.kv_lengths[a];
  for (int i = threadIdx.x; i < kBins; i += kSelThreads) sh.hist[i] = 0;
  __syncthreads();
  if (n < 0 || n > p.m.max_cells) {
    if (g == 0 && threadIdx.x == 0) atomicOr(p.status, KVGQA_FLAG_POSITION_RANGE);
    return;
  }
  // The form goes by the sequence's own length: a server's mass is as wide as the
  // longest context it allows for, whatever its sequences hold.
  if (!WIDE || n <= kCachedCells) select_cells<true>(p, a, g, n, sh, cells);
  else select_cells<false>(p, a, g, n, sh, cells);
}

constexpr int kMoveThreads = 256;
constexpr int kMoveCtas = 4;     // resident on an SM
constexpr int kMoveBatch = 4;    // 16-byte chunks per thread and batch (32 sequences to 2048 cells: 105 us; 2 or 8 chunks 119)
constexpr int kTablePages = 2048;  // pages of the table kept in shared memory (more are looked up in L2)

__global__ void __launch_bounds__(kMoveThreads, kMoveCtas) paged_evict_move_kernel(const __grid_constant__ PagedEvictParams p,
                                                                           int slices) {
  __shared__ int pages[kTablePages];
  int b = blockIdx.x;
  const int slice = b % slices;
  b /= slices;
  uint16_t* cache = b & 1 ? p.v_cache : p.k_cache;
  b >>= 1;
  const int a = b / p.H_kv, g = b % p.H_kv;
  const int shift = p.m.page_shift, page = 1 << shift;
  const int n = p.m.kv_lengths[a];  // (an input of the call, like the table: not written by kernel 1)
  bool ok = n > p.keep && n <= p.m.max_cells;
  const int n_pages = ok ? (n + page - 1) >> shift : 0;
  for (int i = threadIdx.x; i < n_pages; i += kMoveThreads) {
    const int pid = paged_page(p.m, a, i << shift);
    ok = ok && pid >= 0;
    if (i < kTablePages) pages[i] = pid;
  }
  ok = __syncthreads_and(ok);
  // Whether there is anything to move or not: the wait of the kernel behind this
  // one covers this grid alone, and kernel 1 only through the wait in here.
  pdl_wait();
  if (!ok) return;  // uniform
  const int32_t* kept = p.kept + (static_cast<size_t>(a) * p.H_kv + g) * p.keep;
  const int chunks = p.D / 8 / slices;              // 16-byte chunks of a row's slice (a power of two)
  const int step = kMoveThreads / chunks;           // rows that the CTA covers at a time
  const int rows = step * kMoveBatch;               // rows of a batch
  const int chunk = threadIdx.x % chunks, row = threadIdx.x / chunks;
  uint16_t* base = cache + (slice * chunks + chunk) * 8;
  auto at = [&](int cell) {
    const int i = cell >> shift;
    const int pid = i < kTablePages ? pages[i] : paged_page(p.m, a, cell);
    return base + ((static_cast<size_t>(pid) * p.H_kv + g) * page + (cell & (page - 1))) * p.D;
  };
  // Batch k moves the kept cells k * rows + row, + step, ...; -1: none, or one
  // that is in its place already.
  auto sources = [&](int k, int (&from)[kMoveBatch]) {
#pragma unroll
    for (int u = 0; u < kMoveBatch; ++u) {
      const int i = k * rows + row + u * step;
      from[u] = i < p.keep ? kept[i] : -1;
      if (from[u] == i) from[u] = -1;
    }
  };
  auto load = [&](const int (&from)[kMoveBatch], uint4 (&v)[kMoveBatch]) {
#pragma unroll
    for (int u = 0; u < kMoveBatch; ++u)
      if (from[u] >= 0) v[u] = *reinterpret_cast<const uint4*>(at(from[u]));
  };
  int from[kMoveBatch], next[kMoveBatch];
  uint4 x[kMoveBatch], y[kMoveBatch];
  sources(0, from);
  load(from, x);
  sources(1, next);
  const int batches = (p.keep + rows - 1) / rows;
  for (int k = 0; k < batches; ++k) {
    load(next, y);  // batch k + 1
    int after[kMoveBatch];
    sources(k + 2, after);
    __syncthreads();  // every read of batch k's cells, and those batch k overwrites, is done
#pragma unroll
    for (int u = 0; u < kMoveBatch; ++u) {
      if (from[u] >= 0) *reinterpret_cast<uint4*>(at(k * rows + row + u * step)) = x[u];
      x[u] = y[u];
      from[u] = next[u];
      next[u] = after[u];
    }
  }
}

}  // namespace

cudaError_t launch_paged_evict(const PagedEvictParams& p, cudaStream_t stream) {
  const long long heads = static_cast<long long>(p.m.A) * p.H_kv;
  if (heads == 0) return cudaSuccess;
  // Column slices until there are CTAs for four rounds of the GPU, so that
  // sequences of different lengths even out: down to 64 bytes, and to one
  // 32-byte sector where the heads are too few to fill the GPU once.  (32 sequences
  // of 8 heads: 105 us in slices of 64 bytes, longer in ones of 32 or 128.)
  const long long round = static_cast<long long>(p.num_sms) * kMoveCtas;
  int slices = 1;
  while (slices < p.D / 32 && heads * 2 * slices < 4 * round) slices *= 2;
  if (heads * 2 * slices < round) slices *= 2;
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
  cfg.dynamicSmemBytes = static_cast<size_t>(std::min(p.mass_cells, kCachedCells)) * sizeof(float);
  // (without the longer form in the kernel 4 sequences take 6.78-6.81 us, with it 6.84-6.87)
  const cudaError_t e = p.mass_cells > kCachedCells ? cudaLaunchKernelEx(&cfg, paged_evict_select_kernel<true>, p)
                                                    : cudaLaunchKernelEx(&cfg, paged_evict_select_kernel<false>, p);
  if (e != cudaSuccess) return e;
  cfg.dynamicSmemBytes = 0;
  cfg.gridDim = dim3(static_cast<unsigned>(heads * 2 * slices));
  cfg.blockDim = dim3(kMoveThreads);
  return cudaLaunchKernelEx(&cfg, paged_evict_move_kernel, p, slices);
}

}  // namespace kvgqa
