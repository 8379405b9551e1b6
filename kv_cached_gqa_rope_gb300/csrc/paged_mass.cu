// The attention weight that each cell of a paged cache gets from a chunk of
// new tokens, added to what it has so far:
//
//   mass[a, g, j] += sum over tokens n of sequence a that see cell j, heads h of KV head g,
//                    of exp(scale * q[n, h] . k_j - lse[n, h])
//
// lse comes with the attention's output, so the weights need K alone: no
// softmax state, no V.  A cell's sum is over queries, so the scores are laid
// out transposed, S^T = K Q^T with one TMEM lane per cell: each thread adds up
// one cell's weights in registers, and nothing crosses threads until it writes
// its cell.  Every cell is summed by one thread in one order and updated once, so
// the result does not depend on how the work is dealt.
//
// An item is 256 cells of one sequence and KV head (two 128-cell tiles, A and
// B).  The queries of the KV group are its columns, (token, head of the group)
// with the group padded to a power of two, in blocks of 128.  Per item:
//   warp 8      TMA of the two K tiles, one box per page (ring of 2 items, 4 at D = 64);
//   warp 9      TMA of the query blocks (ring) and their log sums, as negated
//               base-2 logs, into shared memory (-inf for columns without a query); a
//               head's blocks stay there for all of its items if they fit the ring;
//   warps 10, 11 S_x^T = K_x Q^T of each block into TMEM (x = A, B, two buffers each);
//   warps 0-3   tile A, warps 4-7 tile B: exp2 of the scaled scores less the
//               column's log sum, added to the cell's sum; at the item's end
//               each thread adds that to its cell (as a reduction in L2: a
//               load would have to be waited for).
// The items are dealt as contiguous equal shares of their column blocks to a
// persistent grid.
//
// What bounds it, as measured (32 query heads, 8 KV heads of 128): single tokens by
// the stream of K and about 5 us of start and end (32 sequences of up to 4095 cells,
// pages of 16: 25.6 us, 5.4 TB/s of cells; with a copy per page and half of a head
// the producer warp was the bound, 27.8 us).  Windows of 64 tokens over 4000-16000
// cells take 50 us (0.79 PFLOP/s, 3.3 TB/s) where the MMAs, the exponentials and the
// stream would each take 17-24: a block of 128 columns costs a softmax warp 1700
// clocks, of which the special-function unit is busy 1024 with both tiles' warps,
// and an item about 1500 of waits and set-up beside its blocks.  Two warps more a
// tile, with their sums joined through shared memory, measured 48 us on windows
// but 28.5 on single tokens; 128 columns in registers at once spill (69).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <mutex>

#include "elem.cuh"
#include "paged.cuh"
#include "paged_tiles.cuh"
#include "tcgen05.cuh"

namespace kvgqa {
namespace {

constexpr int BK = 128;        // cells of a tile (= MMA M = TMEM lanes)
constexpr int ITEM = 2 * BK;   // cells of an item
constexpr int BC = 128;        // columns of a block
constexpr int SUB = 16384;     // one [128 rows x 64 16-bit values] swizzled sub-tile of a query block
constexpr int THREADS = 12 * 32;
constexpr int W_K = 8, W_Q = 9, W_MMA = 10;  // and W_MMA + 1
constexpr int TMEM_COLS = 512; // S^T of A and B, two buffers each, 128 columns
constexpr int kQueryBlocks = 2; // query blocks in flight, or resident
constexpr int NL = 8;          // log-sum slots
constexpr unsigned FULLMASK = 0xffffffffu;

template <int D>
struct MCfg {
  static constexpr int NSUB = D / 64;
  using Tile = PagedTile<D>;
  static constexpr int TILE = Tile::BYTES;          // of cells, or a query block
  static constexpr int NK = D == 128 ? 2 : 4;       // items in flight
  static constexpr int NQ = kQueryBlocks;
  static constexpr int K_OFF = 0;
  static constexpr int Q_OFF = NK * 2 * TILE;
  static constexpr int LSE_OFF = Q_OFF + NQ * TILE;
  static constexpr int SCR_OFF = LSE_OFF + NL * BC * 4;
  // k_full[NK], k_empty[NK], q_full[NQ], q_empty[NQ], l_full[NL], l_empty[NL], s_full[4], s_empty[4], drain
  static constexpr int SEQ_OFF = SCR_OFF + 64 * 4;  // the walk's sequences
  static constexpr int BAR_OFF = SEQ_OFF + kPagedSeqs * sizeof(PagedSeq);
  static constexpr int NBAR = 2 * NK + 2 * NQ + 2 * NL + 10;
  static constexpr int SLOT_OFF = BAR_OFF + NBAR * 8;
  static constexpr int FLAG_OFF = SLOT_OFF + 8;
  static constexpr int SMEM = FLAG_OFF + 16 + 1024;
  static_assert(SMEM <= 232448, "shared memory budget");
  static_assert(SEQ_OFF - SCR_OFF >= paged_scratch_bytes(THREADS), "the schedule's scratch");
};

// Column blocks of a sequence, and the units of its items: one per column
// block and tile pair, one for the item itself.
__device__ __forceinline__ int col_blocks(const PagedMassParams& p, const PagedSeq& s) {
  return ((s.ql << p.gp_shift) + BC - 1) / BC;
}
__device__ __forceinline__ int item_units(const PagedMassParams& p, const PagedSeq& s) {
  return s.ql > 0 ? col_blocks(p, s) + 1 : 0;
}
__device__ __forceinline__ int seq_units(const PagedMassParams& p, const PagedSeq& s) {
  return p.H_kv * ((s.kl + ITEM - 1) / ITEM) * item_units(p, s);
}

// Walks the items whose first unit lies in this CTA's range.
struct MassWalk {
  const PagedMassParams* p;
  const PagedSeq* seqs;
  int a_first, n_seqs;
  int loads;              // query blocks loaded for the heads before this one (before this item, if streamed)
  bool fresh;             // the CTA's first item of this head
  int v, v1;              // the item's first unit, the end of the range
  int a, g, kb;           // sequence, KV head, item of the head
  int first, ql, kl, off, n_items, units, nblk;
  bool ok;

  __device__ __forceinline__ void load_seq() {
    const PagedSeq s = range_seq(p->m, *this, a);
    first = s.first;
    ql = s.ql;
    kl = s.kl;
    off = kl - ql;
    n_items = (kl + ITEM - 1) / ITEM;
    units = item_units(*p, s);
    nblk = col_blocks(*p, s);
  }
  __device__ void advance() {
    if (!resident()) loads += nblk - first_block(0);
    else if (last()) loads += nblk;
    v += units;
    fresh = false;
    if (++kb == n_items) {
      kb = 0;
      fresh = true;
      if (++g == p->H_kv) {
        g = 0;
        do {
          if (++a >= p->m.A) {
            ok = false;
            return;
          }
          load_seq();
        } while (ql == 0);
      }
    }
    ok = v < v1;
  }
  __device__ void init(const PagedMassParams* params, const PagedRange& r) {
    p = params;
    seqs = r.seqs;
    a = r.a;
    a_first = r.first_seq;
    n_seqs = r.n_seqs;
    v1 = r.v1;
    loads = 0;
    fresh = true;
    load_seq();
    const int i = (r.v0 - r.pre + units - 1) / units;  // the first item from v0 on
    v = r.pre + i * units;
    g = i / n_items;
    kb = i % n_items;
    ok = v < v1;
    if (g == p->H_kv) {  // it is the next sequence's
      g = p->H_kv - 1;
      kb = n_items - 1;
      v -= units;
      advance();
      loads = 0;
    }
  }
  // A head's query blocks stay in the ring for all of its items if they fit;
  // else every item streams them through it.
  __device__ __forceinline__ bool resident() const { return nblk <= kQueryBlocks; }
  __device__ __forceinline__ bool last() const { return kb + 1 == n_items || v + units >= v1; }  // of this head, here
  // Cells of tile x of the item.
  __device__ __forceinline__ int live(int x) const { return min(BK, kl - kb * ITEM - x * BK); }
  // The first column block of which some token sees a cell of tile x (the
  // last token sees every cell, so the last block always counts).
  __device__ __forceinline__ int first_block(int x) const {
    const int t = kb * ITEM + x * BK - off;  // the first token that sees the tile
    return t <= 0 ? 0 : (t << p->gp_shift) / BC;
  }
};

// Bits lo .. hi - 1 of 32.
__device__ __forceinline__ uint32_t span_mask(int lo, int hi) {
  const uint32_t below = hi >= 32 ? 0xffffffffu : (1u << max(hi, 0)) - 1u;
  return lo >= 32 ? 0u : below >> max(lo, 0) << max(lo, 0);
}

// Adds the weights of 32 columns to two pairs of sums: exp2 of the scaled scores
// less the columns' log sums.  PICKED: of the columns in the mask alone (what is
// in the others may be anything).
template <bool PICKED>
__device__ __forceinline__ void add_lot(const uint32_t (&u)[32], const float* ls, float2 c2, uint32_t mask, float2& s0,
                                        float2& s1) {
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    const float4 l4 = *reinterpret_cast<const float4*>(ls + i);
    float2 xa = ffma2(make_float2(__uint_as_float(u[i]), __uint_as_float(u[i + 1])), c2, make_float2(l4.x, l4.y));
    float2 xb = ffma2(make_float2(__uint_as_float(u[i + 2]), __uint_as_float(u[i + 3])), c2, make_float2(l4.z, l4.w));
    if (PICKED) {
      xa.x = mask >> i & 1 ? xa.x : -INFINITY;
      xa.y = mask >> (i + 1) & 1 ? xa.y : -INFINITY;
      xb.x = mask >> (i + 2) & 1 ? xb.x : -INFINITY;
      xb.y = mask >> (i + 3) & 1 ? xb.y : -INFINITY;
    }
    s0 = fadd2(s0, make_float2(ex2(xa.x), ex2(xa.y)));
    s1 = fadd2(s1, make_float2(ex2(xb.x), ex2(xb.y)));
  }
}

// The same for a block's columns lo .. hi - 1 (not PICKED: all of them).  Two lots
// in turn, one read from tensor memory while the other's weights are computed; in
// a loop and without a choice inside it, since the whole block unrolled spills and
// a branch per lot keeps the compiler from overlapping them (windows of 64 tokens:
// 50 us; unrolled 52-64, with the choice inside 54).
template <bool PICKED>
__device__ __forceinline__ void add_columns(uint32_t s_tm, const float* ls, float2 c2, int lo, int hi, float2& sum) {
  uint32_t u0[32], u1[32];
  float2 sum1 = make_float2(0.f, 0.f);
  tmem_ld32(s_tm, u0);
#pragma unroll 1
  for (int q = 0; q < (PICKED ? hi : BC); q += 64) {
    tmem_wait_ld();
    tmem_ld32(s_tm + q + 32, u1);
    add_lot<PICKED>(u0, ls + q, c2, PICKED ? span_mask(lo - q, hi - q) : 0, sum, sum1);
    tmem_wait_ld();
    if (q + 64 < BC) tmem_ld32(s_tm + q + 64, u0);
    add_lot<PICKED>(u1, ls + q + 32, c2, PICKED ? span_mask(lo - q - 32, hi - q - 32) : 0, sum, sum1);
  }
  tmem_wait_ld();  // (the read ahead of a short block's last lot)
  sum = fadd2(sum, sum1);
}

template <int D, bool F16>
__global__ void __launch_bounds__(THREADS, 1)
paged_mass_kernel(const __grid_constant__ PagedMassParams p, const __grid_constant__ CUtensorMap map_q,
                  const __grid_constant__ CUtensorMap map_k) {
  using C = MCfg<D>;
  using E = Elem<F16>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                         ~static_cast<uintptr_t>(1023));
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
  uint64_t* k_empty = k_full + C::NK;
  uint64_t* q_full = k_empty + C::NK;
  uint64_t* q_empty = q_full + C::NQ;
  uint64_t* l_full = q_empty + C::NQ;
  uint64_t* l_empty = l_full + NL;
  uint64_t* s_full = l_empty + NL;    // [tile * 2 + buffer]
  uint64_t* s_empty = s_full + 4;
  uint64_t* drain = s_empty + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::SLOT_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::FLAG_OFF);
  float* lse_s = reinterpret_cast<float*>(smem + C::LSE_OFF);  // [NL][BC]
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

  // What needs no input comes before the wait for the previous kernel.
  if (warp == W_K && lane == 0) {
    tma_prefetch_map(&map_q);
    tma_prefetch_map(&map_k);
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NK; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 2);  // both issuers
    }
    for (int s = 0; s < C::NQ; ++s) {
      mbar_init(&q_full[s], 1);
      mbar_init(&q_empty[s], 2);
    }
    for (int s = 0; s < NL; ++s) {
      mbar_init(&l_full[s], 1);
      mbar_init(&l_empty[s], 8);  // every softmax warp, whether its tile uses the block or not
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&s_empty[s], 4);  // one arrival per warp of the tile's group
    }
    mbar_init(&drain[0], 1);
    mbar_init(&drain[1], 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  pdl_wait();
  // Not before the wait: a grid that holds tensor memory while it waits could keep
  // it from the CTAs it waits for.
  if (warp == W_MMA) {
    tmem_alloc(tmem_slot, TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  pdl_trigger();  // the next kernel may set itself up on SMs that are done here
  PagedRange range;
  bool work = paged_range<THREADS>(p.m, p.status, p.num_ctas, 1, reinterpret_cast<int*>(smem + C::SCR_OFF),
                                   reinterpret_cast<PagedSeq*>(smem + C::SEQ_OFF), range,
                                   [&](const PagedSeq& q) { return seq_units(p, q); });
  tc_fence_after();  // (past the barriers of paged_range)
  MassWalk walk;
  if (work) {
    walk.init(&p, range);
    work = walk.ok;
  }
  if (!work) {  // uniform: no item begins in this range
    if (warp == W_MMA) tmem_dealloc(*tmem_slot, TMEM_COLS);
    return;
  }
  const uint32_t tmem = uniform(*tmem_slot);
  const uint32_t sbase = uniform(smem_u32(smem));
#define KVGQA_WAIT(bar, parity) __all_sync(FULLMASK, mbar_wait_bounded((bar), (parity), abort_flag, p.status))

  if (warp == W_K) {
    // ------------------------------------------------------------ K producer
    const uint64_t pol = l2_evict_first_policy();  // each cell is read once
    const int rows = min(1 << p.m.page_shift, BK);
    // box i of an item holds the cells kb * ITEM + i * rows ..; at most 16.  A
    // lane's table entry is read an item ahead within a head.
    auto fetch = [&](int kb) {
      const int cell = kb * ITEM + lane * rows;
      return lane < ITEM / rows && cell < walk.kl ? paged_entry(p.m, walk.a, cell) : 0;
    };
    int it = 0, entry = fetch(walk.kb);
    for (; walk.ok; ++it) {
      const int s = it % C::NK;
      const int n = (min(ITEM, walk.kl - walk.kb * ITEM) + rows - 1) / rows;
      if (it >= C::NK && !KVGQA_WAIT(&k_empty[s], ((it / C::NK) - 1) & 1)) break;
      if (lane < n && (entry < 0 || entry >= p.m.P)) atomicOr(p.status, KVGQA_FLAG_PAGE_RANGE);
      const int group = paged_tile_group(p.m, entry, p.H_kv, walk.g, walk.kb * ITEM + lane * rows);
      if (lane == 0) mbar_arrive_expect_tx(&k_full[s], n * rows * 128 * C::NSUB);
      __syncwarp();
      if (lane < n)
        tma_load_4d(smem + C::K_OFF + s * 2 * C::TILE + lane * rows * 128 * C::NSUB, &map_k, 0, 0, 0, group, &k_full[s], pol);
      walk.advance();
      if (walk.ok) entry = fetch(walk.kb);
    }
    __syncwarp();
    if (*abort_flag) {
      volatile int none = 0;
      for (int t = it - C::NK < 0 ? 0 : it - C::NK; t < it; ++t)
        mbar_wait_bounded(&k_full[t % C::NK], (t / C::NK) & 1, &none, nullptr);
    }
  } else if (warp == W_Q) {
    // ------------------------------------------------------------ queries and log sums
    const uint64_t pol = l2_evict_last_policy();
    const int gp = 1 << p.gp_shift;
    int n = 0;  // blocks so far
    bool ok = true;
    for (; walk.ok && ok; walk.advance()) {
      if (walk.resident() && !walk.fresh) continue;
      for (int blk = walk.resident() ? 0 : walk.first_block(0); blk < walk.nblk; ++blk, ++n) {
        const int tok0 = (blk * BC) >> p.gp_shift;
        const int s = n % C::NQ;
        ok = n < C::NQ || KVGQA_WAIT(&q_empty[s], ((n / C::NQ) - 1) & 1);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&q_full[s], p.box_tokens * gp * 128 * C::NSUB);
          for (int sub = 0; sub < C::NSUB; ++sub)
            tma_load_4d(smem + C::Q_OFF + s * C::TILE + sub * SUB, &map_q, sub * 64, 0, walk.g, walk.first + tok0,
                        &q_full[s], pol);
        }
        __syncwarp();
        // log sums of this lane's 4 columns, in base 2 and negated
        float ls[BC / 32];
#pragma unroll
        for (int i = 0; i < BC / 32; ++i) {
          const int col = lane + 32 * i, t = tok0 + (col >> p.gp_shift), h = col & (gp - 1);
          ls[i] = -INFINITY;
          if (t < walk.ql && h < p.G)
            ls[i] = p.lse[static_cast<size_t>(walk.first + t) * p.H_q + walk.g * p.G + h] * -1.4426950408889634f;
        }
        ok = n < NL || KVGQA_WAIT(&l_empty[n % NL], ((n / NL) - 1) & 1);
        if (!ok) {
          ++n;  // (its query block is on the way)
          break;
        }
#pragma unroll
        for (int i = 0; i < BC / 32; ++i) lse_s[(n % NL) * BC + lane + 32 * i] = ls[i];
        __syncwarp();
        if (lane == 0) mbar_arrive(&l_full[n % NL]);
      }
    }
    __syncwarp();
    if (*abort_flag) {
      volatile int none = 0;
      for (int t = n - C::NQ < 0 ? 0 : n - C::NQ; t < n; ++t)
        mbar_wait_bounded(&q_full[t % C::NQ], (t / C::NQ) & 1, &none, nullptr);
    }
  } else if (warp >= W_MMA) {
    // ------------------------------------------------------------ MMA issuers, one per tile
    const int x = uniform(warp - W_MMA);
    int it = 0, sn = 0;
    bool ok = true, issued = false;
    for (; walk.ok && ok; walk.advance(), ++it) {
      const int ks = it % C::NK;
      const bool resident = walk.resident();
      if (!KVGQA_WAIT(&k_full[ks], (it / C::NK) & 1)) break;
      const int fb0 = walk.first_block(0), fb = walk.live(x) > 0 ? walk.first_block(x) : walk.nblk;
      if (resident && walk.fresh)
        for (int n = walk.loads; n < walk.loads + walk.nblk && ok; ++n) ok = KVGQA_WAIT(&q_full[n % C::NQ], (n / C::NQ) & 1);
      if (!ok) break;
      const uint32_t k_lo = smem_desc_lo(uniform(sbase + C::K_OFF + (ks * 2 + x) * C::TILE), 16);
      for (int blk = fb0; blk < walk.nblk; ++blk) {
        const int n = walk.loads + (resident ? blk : blk - fb0), qs = n % C::NQ;
        if (!resident) ok = KVGQA_WAIT(&q_full[qs], (n / C::NQ) & 1);
        if (!ok) break;
        if (blk >= fb) {
          const int buf = x * 2 + (sn & 1);
          // only the columns that hold a query, in whole groups of 16
          const int cols = min(BC, (walk.ql << p.gp_shift) - blk * BC);
          const uint32_t idesc = uniform(idesc_f16kind_f32(E::kMmaFormat, BK, (cols + 15) & ~15, 0));
          const uint32_t q_lo = smem_desc_lo(uniform(sbase + C::Q_OFF + qs * C::TILE), 16);
          const uint32_t s_tm = uniform(tmem + buf * BC);
          if (sn >= 2) {
            ok = KVGQA_WAIT(&s_empty[buf], ((sn >> 1) - 1) & 1);
            if (!ok) break;
          }
          ++sn;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t o = (kk % 4) * (32 >> 4);
              umma_f16_ss_lo<C::Tile::GROUP, 1024>(s_tm, k_lo + (kk / 4) * (1024 >> 4) + o, q_lo + (kk / 4) * (SUB >> 4) + o,
                                                     idesc, kk > 0);
            }
            umma_commit(&s_full[buf]);
          }
          __syncwarp();
          issued = true;
        }
        if (!resident) {
          if (elect_one()) umma_commit(&q_empty[qs]);
          __syncwarp();
        }
      }
      if (!ok) break;
      if (elect_one()) {
        umma_commit(&k_empty[ks]);
        if (resident && walk.last())
          for (int n = walk.loads; n < walk.loads + walk.nblk; ++n) umma_commit(&q_empty[n % C::NQ]);
      }
      __syncwarp();
    }
    if (*abort_flag && issued) {
      if (elect_one()) umma_commit(&drain[x]);
      __syncwarp();
      volatile int none = 0;
      mbar_wait_bounded(&drain[x], 0, &none, nullptr);
    }
  } else {
    // ------------------------------------------------------------ weights (warps 0-7)
    const int x = warp >> 2;           // tile A or B
    const int r = threadIdx.x & 127;   // cell of the tile == TMEM lane
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const float2 c2 = make_float2(p.scale_log2, p.scale_log2);
    int sn = 0;  // column blocks of this tile so far
    bool ok = true;
    // The log sums of load n are there; they are done with.
    auto take = [&](int n) {
      ok = ok && __all_sync(FULLMASK, mbar_wait_bounded(&l_full[n % NL], (n / NL) & 1, abort_flag, p.status));
    };
    auto pass = [&](int n) {
      __syncwarp();
      if (lane == 0) mbar_arrive(&l_empty[n % NL]);
    };
    for (; walk.ok && ok; walk.advance()) {
      const int live = walk.live(x), fb0 = walk.first_block(0);
      const bool resident = walk.resident();
      if (resident && walk.fresh)
        for (int n = walk.loads; n < walk.loads + walk.nblk; ++n) take(n);
      // Streamed blocks that this tile does not use are passed on.
      const int fb = live > 0 ? walk.first_block(x) : walk.nblk;
      if (!resident)
        for (int n = walk.loads; n < walk.loads + fb - fb0 && ok; ++n) {
          take(n);
          pass(n);
        }
      if (!ok) break;
      if (live > 0) {
        const int cell = walk.kb * ITEM + x * BK + r;
        float* dst = p.mass + (static_cast<size_t>(walk.a) * p.H_kv + walk.g) * p.mass_cells + cell;
        // column i of block blk sees this cell iff blk * BC + i >= c_min
        const int c_min = max(cell - walk.off, 0) << p.gp_shift;
        const int c_tile = max(walk.kb * ITEM + x * BK + live - 1 - walk.off, 0) << p.gp_shift;  // the tile's largest
        float2 sum = make_float2(0.f, 0.f);
        for (int blk = fb; blk < walk.nblk; ++blk, ++sn) {
          const int buf = x * 2 + (sn & 1), n = walk.loads + (resident ? blk : blk - fb0);
          ok = __all_sync(FULLMASK, mbar_wait_bounded(&s_full[buf], (sn >> 1) & 1, abort_flag, p.status));
          if (!resident) take(n);
          if (!ok) break;
          tc_fence_after();
          const float* ls = lse_s + (n % NL) * BC;
          const int cols = min(BC, (walk.ql << p.gp_shift) - blk * BC);
          const uint32_t s_tm = tmem + lane_base + buf * BC;
          const int lo = c_min - blk * BC;
          if (cols <= 16) {  // single tokens: their heads alone
            uint32_t u[16];
            tmem_ld16(s_tm, u);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float w = ex2(fmaf(__uint_as_float(u[i]), p.scale_log2, ls[i]));
              sum.x += i >= lo && i < cols ? w : 0.f;
            }
          } else if (cols == BC && blk * BC >= c_tile) {  // every column, by every cell of the tile
            add_columns<false>(s_tm, ls, c2, 0, BC, sum);
          } else {
            add_columns<true>(s_tm, ls, c2, lo, cols, sum);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_empty[buf]);
          if (!resident) pass(n);
        }
        if (!ok) break;
        if (r < live) atomicAdd(dst, sum.x + sum.y);  // the cell's only update in this call: nothing to wait for
      }
      if (resident && walk.last())
        for (int n = walk.loads; n < walk.loads + walk.nblk; ++n) pass(n);
    }
  }
#undef KVGQA_WAIT

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == W_MMA) tmem_dealloc(tmem, TMEM_COLS);
}

template <int D, bool F16>
cudaError_t launch_d(const PagedMassParams& p, const CUtensorMap& mq, const CUtensorMap& mk, cudaStream_t stream) {
  static std::once_flag flags[64];
  static cudaError_t errs[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::call_once(flags[dev], [&] {
    errs[dev] = cudaFuncSetAttribute(paged_mass_kernel<D, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     MCfg<D>::SMEM);
  });
  if (errs[dev] != cudaSuccess) return errs[dev];
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.num_ctas);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = MCfg<D>::SMEM;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_mass_kernel<D, F16>, p, mq, mk);
}

}  // namespace

cudaError_t launch_paged_mass(const PagedMassParams& params, cudaStream_t stream) {
  if (params.m.A == 0 || params.m.N == 0) return cudaSuccess;
  PagedMassParams p = params;
  p.gp_shift = 0;
  while ((1 << p.gp_shift) < p.G) ++p.gp_shift;
  const int gp = 1 << p.gp_shift;
  // A block's box holds no more tokens than any sequence has (in a power of
  // two, and whole 8-row groups of the swizzle): a single token's block is its
  // own heads, not 128 rows of its neighbours.
  p.box_tokens = 1;
  while (p.box_tokens * gp < BC && (p.box_tokens < p.m.max_query_len || p.box_tokens * gp < 8)) p.box_tokens *= 2;
  auto enc = tma_encoder();
  if (!enc) return cudaErrorNotSupported;
  const CUtensorMapDataType type = p.f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const cuuint64_t D = p.D, G = p.G, Hkv = p.H_kv;
  const cuuint32_t es[4] = {1, 1, 1, 1};
  CUtensorMap mq, mk;
  {
    const cuuint64_t dims[4] = {D, G, Hkv, static_cast<cuuint64_t>(p.m.N)};
    const cuuint64_t strides[3] = {D * 2, D * 2 * G, D * 2 * G * Hkv};
    const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(gp), 1, static_cast<cuuint32_t>(p.box_tokens)};
    if (enc(&mq, type, 4, const_cast<uint16_t*>(p.q), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  if (paged_tile_map(enc, &mk, type, p.k_cache, p.D, p.m.P, p.H_kv, p.m.page_shift) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  if (p.D == 128) return p.f16 ? launch_d<128, true>(p, mq, mk, stream) : launch_d<128, false>(p, mq, mk, stream);
  if (p.D == 64) return p.f16 ? launch_d<64, true>(p, mq, mk, stream) : launch_d<64, false>(p, mq, mk, stream);
  return cudaErrorInvalidValue;
}

}  // namespace kvgqa
