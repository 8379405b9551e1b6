// The paged cache as the kernels see it: the packed new tokens of A sequences,
// their cells, and the block table that maps a sequence's cell to a page of
// the pool [P, H_kv, page, D].  Internal to libkvgqa.
#pragma once

#include <cstdint>

#include "kvgqa.h"
#include "kvgqa_internal.h"

namespace kvgqa {

// What a sequence's metadata says, after the checks that only the device can
// make.  `ok` is false for metadata out of range: such a sequence is skipped.
struct PagedSeq {
  int first;  // its first row in the packed tokens
  int ql;     // new tokens
  int kl;     // cells, the new tokens' included
  bool ok;
};

__device__ __forceinline__ PagedSeq paged_seq(const PagedMeta& m, int a) {
  PagedSeq s;
  s.first = m.query_starts[a];
  const int end = m.query_starts[a + 1];
  s.kl = m.kv_lengths[a];
  s.ok = s.first >= 0 && end >= s.first && end <= m.N && end - s.first <= m.max_query_len && s.kl >= end - s.first &&
         s.kl <= m.max_cells;
  s.ql = s.ok && end - s.first >= m.tokens_lo && end - s.first <= m.tokens_hi ? end - s.first : 0;
  return s;
}

// Page of cell `cell` of sequence a, or -1 where the table's entry is no page
// of the pool.
__device__ __forceinline__ int paged_page(const PagedMeta& m, int a, int cell) {
  const int pid = m.block_table[static_cast<size_t>(a) * m.max_pages + (cell >> m.page_shift)];
  return pid >= 0 && pid < m.P ? pid : -1;
}

// The share of a CTA in a persistent grid: the range [v0, v1) of virtual units,
// w to a CTA, and the sequence `a` that v0 falls in, whose units begin at `pre`.
// Every CTA computes the same prefix sums from the metadata, so there is no
// planning kernel and no plan to keep.
struct PagedRange {
  int v0, v1, w, a, pre;
  const PagedSeq* seqs;  // sequences first_seq .. + n_seqs - 1, read once for the CTA
  int first_seq, n_seqs;
};
constexpr int kPagedSeqs = 32;  // sequences whose metadata a CTA keeps at hand

// The host refuses calls whose units could reach this many, but counts every
// packed row once.  Sequences whose rows overlap (query_starts that fall and rise
// again) can pass it together, so sums of units stop there instead of wrapping;
// one sequence's units are below it.
constexpr int kPagedUnits = 1 << 30;
__device__ __forceinline__ int add_units(int x, int y) {
  return static_cast<int>(min(static_cast<unsigned>(x) + static_cast<unsigned>(y), static_cast<unsigned>(kPagedUnits)));
}

// The scratch of paged_range in shared memory: each warp's sum and the range's
// first sequence with its prefix; in whole groups of 16 bytes.
constexpr int paged_scratch_bytes(int threads) { return (threads / 32 + 2 + 3) / 4 * 16; }

// Called by the whole CTA of THREADS; units(seq) gives a sequence's units,
// scratch has paged_scratch_bytes(THREADS) and seqs kPagedSeqs entries of shared
// memory, which must not overlap: the entries are written while the scratch is read.
// False if nothing is left for this CTA, and for every CTA if the sequences have
// kPagedUnits or more together.  Passes a barrier of the CTA in either case (m.A > 0).
template <int THREADS, typename Units>
__device__ bool paged_range(const PagedMeta& m, int32_t* status, int num_ctas, int min_units, int* scratch,
                            PagedSeq* seqs, PagedRange& r, Units units_of) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int NW = THREADS / 32;
  // Prefix sums over chunks of one sequence per thread.  The last chunk's stay
  // in registers: with no more sequences than threads that is all there is.
  int units = 0, excl = 0, total = 0;
  bool bad = false;
  const int chunks = (m.A + THREADS - 1) / THREADS;
  auto scan = [&](int chunk) {
    const int a = chunk * THREADS + tid;
    units = 0;
    if (a < m.A) {
      const PagedSeq s = paged_seq(m, a);
      bad = bad || !s.ok;
      units = units_of(s);
      if (m.A <= kPagedSeqs) seqs[a] = s;
    }
    int incl = units;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl = add_units(incl, t);
    }
    if (chunk > 0) __syncthreads();  // the last chunk's sums have been read
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    excl = add_units(total, incl - units);  // (exact unless the total reaches kPagedUnits)
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const int t = scratch[w];
      if (w < warp) excl = add_units(excl, t);
      total = add_units(total, t);
    }
  };
  for (int c = 0; c < chunks; ++c) scan(c);
  if (blockIdx.x == 0 && (bad || total >= kPagedUnits)) atomicOr(status, KVGQA_FLAG_POSITION_RANGE);
  if (total >= kPagedUnits) return false;
  r.w = max((total + num_ctas - 1) / num_ctas, min_units);
  const long long v0 = static_cast<long long>(blockIdx.x) * r.w;
  if (v0 >= total) return false;
  r.v0 = static_cast<int>(v0);
  r.v1 = min(r.v0 + r.w, total);
  int* found = scratch + NW;
  if (chunks == 1) {
    if (units > 0 && excl <= r.v0 && r.v0 < excl + units) {
      found[0] = tid;
      found[1] = excl;
    }
  } else {
    total = 0;
    __syncthreads();
    for (int c = 0; c < chunks; ++c) {
      scan(c);
      if (units > 0 && excl <= r.v0 && r.v0 < excl + units) {
        found[0] = c * THREADS + tid;
        found[1] = excl;
      }
    }
  }
  __syncthreads();
  r.a = found[0];
  r.pre = found[1];
  r.seqs = seqs;
  r.first_seq = 0;
  r.n_seqs = m.A;
  if (m.A > kPagedSeqs) {  // the table holds the first of this CTA's
    r.first_seq = r.a;
    r.n_seqs = min(kPagedSeqs, m.A - r.a);
    if (tid < r.n_seqs) seqs[tid] = paged_seq(m, r.a + tid);
    __syncthreads();
  }
  return true;
}

// Sequence a of a walk that keeps the range's table.
template <typename Walk>
__device__ __forceinline__ PagedSeq range_seq(const PagedMeta& m, const Walk& w, int a) {
  return a - w.a_first < w.n_seqs ? w.seqs[a - w.a_first] : paged_seq(m, a);
}

}  // namespace kvgqa
