// Grouped-query attention of a chunk of new tokens over a paged cache, on
// tcgen05 tensor cores with the accumulators in tensor memory.
//
//   out[n, h] = sum_j softmax_j(scale * q[n, h] . k_j) v_j,  j = 0 .. the cell of token n
//   lse[n, h] = log sum_j exp(scale * q[n, h] . k_j)
//
// Work.  The query heads of a KV group read the same keys, so a query tile is
// 128 rows of (token, head of the group): 128 / GP tokens of one KV head (GP:
// the group size padded to a power of two; the tensor map fills the padding
// with zeros).  A segment (a, g, b) is block b of two such tiles (A and B) of
// sequence a and KV head g; both read each 128-key tile that is staged in
// shared memory, which is walked from cell 0 to the block's last token.  The
// segments lie one behind the other in a virtual space of units (about one per
// key tile, one for a segment's start and end), of which every CTA of the
// persistent grid (one per SM) takes an equal range: long prompts, short chunks
// and single tokens share one schedule, whose shares differ by a few units.  A
// segment cut by a CTA boundary leaves FP32 partials (m, l, O) of the rows it
// really has, merged by the kernel launched behind this one (in the SMALL form by
// an idle warp of the CTA that finishes the segment's last part: one launch).
//
// Per key tile:
//   warp 8      TMA of the query tiles and the K tile, one box per page (a tile
//               takes 128 / page boxes, issued side by side by as many lanes,
//               each with its page's table entry, read a tile ahead);
//   warp 9      the same for the V tile; in a sequence's last tile it zeroes the
//               rows behind the last cell, which may hold anything (a zero
//               weight times a NaN is a NaN);
//   warps 10, 11 issue tcgen05.mma for A and for B: S_x = Q_x K^T into TMEM
//               and O_x += P_x V with P_x read from TMEM;
//   warps 0-3   softmax of tile A, warps 4-7 of tile B, one thread per row: FP32
//               online softmax (the base follows the row maximum only when it
//               grew by more than 2^8; O / l stays exact), P in the storage type
//               written back over the S columns.  P's rounding is that of the
//               tensor cores' operand type; the sum l is of the unrounded FP32
//               weights.
// While one tile's softmax works on its scores, the other tile's MMAs run.  A
// block of at most 128 rows (a decode step, a short chunk, a prompt's last
// tokens) has no tile B: there the two groups take the key tiles in turn, each
// with its own running maximum, sum and accumulator, which group A joins at the
// end; warps without a row of the sequence skip the softmax.
// What bounds it, as measured (32 query heads, 8 KV heads of 128, BF16):
//   long contexts of single tokens by the stream of K and V: 8 sequences of 65536
//   cells take 260-263 us, 6.7 TB/s, the rate of a copy; shorter ones by that and about
//   12 us of start and end that do not shrink with the cache: 32 sequences of up
//   to 4095 cells 57 us, 4.7 TB/s; 4 of up to 500 cells 8.5-8.7 us, all latency
//   (schedule 2, first tile 1.2, softmax 1.1, P.V and its commit 1.6, epilogue 0.9);
//   long chunks by the chain S -> softmax -> P.V of a tile beside the other
//   tile's MMAs: 4 chunks of 2048 tokens after 6000-14000 cells 1073-1099 us, 1.33-1.36
//   PFLOP/s, a round of two tiles 3300 clocks of which the MMAs take 2048.
//   Measured and not kept: every second or third pair of exponentials as a polynomial
//   (chunks 1513-1970 us where 1304 without), four softmax warpgroups (spills,
//   2795 us), other register splits (1322-1358 against 1301), strict turns of the
//   two issuers (1123 against 1115).
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

constexpr int BM = 128;        // rows of a query tile
constexpr int BN = 128;        // keys of a tile
constexpr int ROWS = 2 * BM;   // rows of a segment's block: tiles A and B
constexpr int SUB = 16384;     // one [128 rows x 64 16-bit values] swizzled sub-tile of a query tile
constexpr int THREADS = 12 * 32;
constexpr int W_K = 8, W_V = 9, W_MMA = 10;  // and W_MMA + 1
// Register split (setmaxnreg): the launch gives every thread kLaunchRegs; the
// role warpgroup drops to kRoleRegs so that the two softmax warpgroups can
// hold a whole score row each.
constexpr int kLaunchRegs = 168, kRoleRegs = 72, kSoftmaxRegs = 216;
static_assert(2 * 128 * kSoftmaxRegs + 128 * kRoleRegs <= THREADS * kLaunchRegs, "register split");
constexpr int TMEM_COLS = 512; // S_A, S_B, O_A, O_B: 128 columns each
constexpr int UNITS_MIN = 4;   // fewest units a CTA is given
constexpr int kSmallRows = 32; // rows of a block in the SMALL form (one warp's)
constexpr unsigned FULLMASK = 0xffffffffu;

// A segment cut at a CTA boundary, noted by the CTA where it starts.
struct PagedCut {
  int rows;    // rows of its block, 0: this CTA starts no cut segment
  int tok;     // first packed token
  int g;       // KV head
  int last;    // last CTA that holds a part of it
  int done;    // SMALL: parts finished so far (zero between calls)
  int pad[3];
};
// One partial result: O as [D / 4][ROWS] groups of 4 values (a thread holds a
// row, so a warp's stores are whole lines), then m[ROWS], then l[ROWS]; slot
// 2b + 1 of CTA b holds a segment that starts there, slot 2b one that started before.
__host__ __device__ constexpr size_t slot_floats(int D) { return static_cast<size_t>(ROWS) * (D + 2); }

// SMALL: no block of the call has more than kSmallRows rows (decode steps, a
// few tokens per sequence), so the stream of K and V is all there is to it.  The
// query buffers hold those rows alone, the output needs no staging, and the
// shared memory that leaves deepens the K and V rings.  (The tensor cores read
// 128 rows from a query buffer's start on; those behind it are whatever lies
// there, and no row sees another.)
template <int D, bool SMALL>
struct ACfg {
  static constexpr int NSUB = D / 64;
  using Tile = PagedTile<D>;
  static constexpr int TILE = Tile::BYTES;          // one K or V tile
  static constexpr int QSUB = SMALL ? kSmallRows * 128 : SUB;
  static constexpr int QTILE = NSUB * QSUB;         // one query tile
  static constexpr int NK = 2 * 128 / D;            // K stages
  static constexpr int NV = (SMALL ? 4 : 2) * 128 / D;  // V stages (a V tile is held longer: through the softmax)
  static_assert(NK % 2 == 0 && NV % 2 == 0, "a stage's tiles alternate with the groups (see the walk)");
  static constexpr int Q_OFF = 0;                   // two query buffers
  static constexpr int K_OFF = 2 * QTILE;
  static constexpr int V_OFF = K_OFF + NK * TILE;
  static constexpr int STG = SMALL ? 0 : 32 * 128;  // output staging of one softmax warp
  static constexpr int STG_OFF = V_OFF + NV * TILE;
  static constexpr int ML_OFF = STG_OFF + 8 * STG;  // group B's m and l of a shared block (and the schedule's scratch)
  static constexpr int SEQ_OFF = ML_OFF + 2 * BM * 4;  // the walk's sequences
  static constexpr int BAR_OFF = SEQ_OFF + kPagedSeqs * sizeof(PagedSeq);
  // q_full[2], q_empty[2], k_full[NK], k_empty[NK], v_full[NV], v_empty[NV],
  // s_full[2], p_full[2], o_done[2], v_land, ml_full, ml_done, part_full[2], drain[2] (index [2] = tile A / B)
  static constexpr int NBAR = 4 + 2 * NK + 2 * NV + 13;
  static constexpr int SLOT_OFF = BAR_OFF + NBAR * 8;
  static constexpr int FLAG_OFF = SLOT_OFF + 8;
  static constexpr int SMEM = FLAG_OFF + 16 + 1024;  // + alignment slack
  static_assert(SMEM <= 232448, "shared memory budget");
};

// ------------------------------------------------------------------ schedule
__device__ __forceinline__ int block_tokens(const PagedAttentionParams& p) { return ROWS >> p.gp_shift; }
// Virtual units: kPair per key tile of a block with both query tiles, one per
// key tile of a block with one, p.end_units for a segment's start and end
// (measured per CTA of a mixed step: 1.74, 1.07 and 4.1 us; of a small call,
// where the stream of K and V is the bound: 1.25 and 1.9 us; finer weights, 3:2:6
// to 7:4:16, come out level over 8 mixed steps).  A sequence's last
// block counts its key tiles; the others, all with two query tiles, count
// off / BN + 1 + ceil((b + 1) tokens / BN) of them, at least what they have, for
// off cells before the new tokens: a form whose sums over blocks are closed.  A
// last block's units are a multiple of a CTA's fewest, so that few short segments
// are dealt whole, one to a CTA (4 requests of up to 500 cells: 8.5 us, cut 11.2; more
// long segments than CTAs lose by it: 32 of up to 4095 cells in 8 heads 54.7 us, cut
// 54.0, mixed steps of 28 sequences 92.4, cut 90.6).
constexpr int kPair = 2;
__device__ __forceinline__ int block_weight(const PagedAttentionParams& p, int ql, int b) {
  return (ql - b * block_tokens(p)) << p.gp_shift > BM ? kPair : 1;
}
// The units of block b of a sequence with ql new tokens.
__device__ __forceinline__ int seg_units(const PagedAttentionParams& p, int off, int ql, int b) {
  const int end = (b + 1) * block_tokens(p);
  return end < ql ? kPair * (off / BN + 1 + (end + BN - 1) / BN) + p.end_units
                  : (block_weight(p, ql, b) * ((off + ql + BN - 1) / BN) + p.end_units + UNITS_MIN - 1) / UNITS_MIN * UNITS_MIN;
}
// The units of a sequence's first n blocks, none of them its last.
__device__ __forceinline__ int pair_units(const PagedAttentionParams& p, int off, int n) {
  int s;  // the sum of ceil(i tokens / BN) over i = 1 .. n
  if (p.gp_shift == 0) {
    s = n * (n + 1);                           // 256 tokens a block: 2i
  } else {
    const int sh = p.gp_shift - 1, m = n >> sh, r = n & ((1 << sh) - 1);
    s = ((m * (m + 1)) >> 1 << sh) + r * (m + 1);  // 2^sh blocks to a key tile: ceil(i / 2^sh)
  }
  return kPair * (n * (off / BN + 1) + s) + p.end_units * n;
}
// The units of one KV head of a sequence.
__device__ __forceinline__ int head_units(const PagedAttentionParams& p, int ql, int off) {
  if (ql == 0) return 0;
  const int b = (ql - 1) / block_tokens(p);  // the last block
  return pair_units(p, off, b) + seg_units(p, off, ql, b);
}
__device__ __forceinline__ int seq_units(const PagedAttentionParams& p, const PagedSeq& s) {
  return p.H_kv * head_units(p, s.ql, s.kl - s.ql);
}

// Walks the key tiles of this CTA's range, segment by segment; every role
// runs its own copy.
struct PagedWalk {
  const PagedAttentionParams* p;
  const PagedSeq* seqs;
  int a_first, n_seqs;
  int v0, v1;
  int a, g, b, nblk;      // segment: sequence, KV head, block of the sequence's nblk
  int first, ql, off;     // the sequence's first packed row, new tokens, cells before them
  int vlo, tiles, kend;   // the segment's virtual start, key tiles, last cell + 1
  int weight;             // units of a key tile
  int j, j_first, j_end;  // key tile, and this CTA's part of the segment
  int ring, slot;         // key tiles before this one; a block without tile B: its query buffer
  bool ok;

  __device__ __forceinline__ void load_seq() {
    const PagedSeq s = range_seq(p->m, *this, a);
    first = s.first;
    ql = s.ql;
    off = s.kl - s.ql;
    const int tb = block_tokens(*p);
    nblk = (ql + tb - 1) / tb;
  }
  __device__ __forceinline__ bool enter() {
    kend = off + min(ql, (b + 1) * block_tokens(*p));
    tiles = (kend + BN - 1) / BN;
    weight = block_weight(*p, ql, b);
    // the key tiles whose first unit lies in [v0, v1)
    const int lo = max(v0 - vlo, 0), hi = v1 - vlo;
    j = j_first = weight == 1 ? lo : (lo + kPair - 1) / kPair;
    j_end = min(tiles, weight == 1 ? hi : (hi + kPair - 1) / kPair);
    return j < j_end;
  }
  __device__ bool next_segment() {
    for (;;) {
      vlo += seg_units(*p, off, ql, b);
      if (vlo >= v1) return false;
      if (++b == nblk) {
        b = 0;
        if (++g == p->H_kv) {
          g = 0;
          do {
            if (++a >= p->m.A) return false;
            load_seq();
          } while (ql == 0);
        }
      }
      if (enter()) return true;
    }
  }
  __device__ void init(const PagedAttentionParams* params, const PagedRange& r) {
    p = params;
    seqs = r.seqs;
    a = r.a;
    a_first = r.first_seq;
    n_seqs = r.n_seqs;
    v0 = r.v0;
    v1 = r.v1;
    load_seq();
    int rem = v0 - r.pre;
    const int head = head_units(*p, ql, off);
    g = rem / head;
    rem -= g * head;
    int lo = 0, hi = nblk - 1;  // the block whose units hold v0
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pair_units(*p, off, mid) <= rem) lo = mid;
      else hi = mid - 1;
    }
    b = lo;
    vlo = v0 - rem + pair_units(*p, off, b);
    ring = slot = 0;
    ok = enter() || next_segment();
  }
  __device__ __forceinline__ bool fresh() const { return j == j_first; }
  // Whether the block has rows in tile B.  If not, the two groups take turns
  // with its key tiles: the group is the parity of the tile's place in the rings,
  // so that with an even number of stages a stage's tiles of such blocks are all
  // of one group.
  __device__ __forceinline__ bool dual() const { return weight != 1; }
  __device__ __forceinline__ int parts() const { return j_end - j_first; }  // key tiles of this part
  __device__ __forceinline__ bool whole() const { return parts() == tiles; }
  __device__ __forceinline__ int last_unit() const { return vlo + weight * (tiles - 1); }
  __device__ __forceinline__ int tok0() const { return b * block_tokens(*p); }
  __device__ __forceinline__ int group() const { return ring & 1; }
  // The next key tile.
  __device__ __forceinline__ void advance() {
    ++ring;
    if (j < j_end - 1) {
      ++j;
    } else {
      if (!dual()) slot ^= 1;
      ok = next_segment();
    }
  }
  // The next segment, from the first key tile of this one (softmax groups, MMA issuers).
  __device__ __forceinline__ void advance_segment() {
    ring += parts();
    if (!dual()) slot ^= 1;
    ok = next_segment();
  }
};

// The TMA boxes of the walk's K or V tile: lane i < n takes the cells from
// j * BN + i * rows on.  A lane's table entry is read one tile ahead within a
// segment: its latency (700 clocks) would stand before every tile's copy.
struct TileBoxes {
  int rows, n;    // cells of a box; boxes of the tile
  int entry;      // this lane's table entry, of tile j
  int j;
  __device__ __forceinline__ void fetch(const PagedWalk& w, int lane, int tile) {
    j = tile;
    const int cell = tile * BN + lane * rows;
    entry = 0;
    if (lane < BN / rows && cell < w.kend) entry = paged_entry(w.p->m, w.a, cell);
  }
  // Of a segment's first tile.
  __device__ __forceinline__ void start(const PagedWalk& w, int lane) {
    rows = min(1 << w.p->m.page_shift, BN);
    fetch(w, lane, w.j);
  }
  // This lane's group of rows in the pool.
  __device__ __forceinline__ int group(const PagedWalk& w, int lane) {
    n = (min(BN, w.kend - w.j * BN) + rows - 1) / rows;
    if (lane < n && (entry < 0 || entry >= w.p->m.P)) atomicOr(w.p->status, KVGQA_FLAG_PAGE_RANGE);
    return paged_tile_group(w.p->m, entry, w.p->H_kv, w.g, w.j * BN + lane * rows);
  }
};

// Atomic add with release and acquire semantics at GPU scope.
__device__ __forceinline__ int atomic_add_acq_rel_gpu(int* ptr, int v) {
  int old;
  asm volatile("atom.add.acq_rel.gpu.s32 %0, [%1], %2;" : "=r"(old) : "l"(ptr), "r"(v) : "memory");
  return old;
}

// One warp merges the parts b0 .. b1 of a block of `rows` <= 32 rows (read past
// L1) and writes out and lse.  Up to 8 lanes share a row, each taking 16 of its
// values at a time.
template <int D, bool F16>
__device__ __forceinline__ void merge_small(const PagedAttentionParams& p, int tok0, int rows, int g, int b0, int b1) {
  using E = Elem<F16>;
  const int lane = threadIdx.x & 31;
  const int share = rows > 16 ? 1 : rows > 8 ? 2 : rows > 4 ? 4 : 8;
  const int row = lane / share, col0 = lane % share * 16;
  const int gi = row & ((1 << p.gp_shift) - 1);
  if (row >= rows || gi >= p.G) return;
  const float* slot0 = p.partials + (static_cast<size_t>(b0) * 2 + 1) * slot_floats(D);
  auto part = [&](int b) { return b == b0 ? slot0 : p.partials + static_cast<size_t>(b) * 2 * slot_floats(D); };
  float M = -INFINITY;
#pragma unroll 4
  for (int b = b0; b <= b1; ++b) M = fmaxf(M, __ldcg(part(b) + ROWS * D + row));
  const size_t head = static_cast<size_t>(tok0 + (row >> p.gp_shift)) * p.H_q + g * p.G + gi;
  for (int col = col0; col < D; col += share * 16) {
    float l = 0.f, acc[16] = {};
#pragma unroll 2
    for (int b = b0; b <= b1; ++b) {
      const float* s = part(b);
      const float m = __ldcg(s + ROWS * D + row), lb = __ldcg(s + ROWS * D + ROWS + row);
      float4 o[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) o[k] = __ldcg(reinterpret_cast<const float4*>(s) + (col / 4 + k) * ROWS + row);
      if (m == -INFINITY) continue;  // this part saw none of the row's cells
      const float w = exp2f(m - M);
      l += w * lb;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        acc[4 * k] += w * o[k].x;
        acc[4 * k + 1] += w * o[k].y;
        acc[4 * k + 2] += w * o[k].z;
        acc[4 * k + 3] += w * o[k].w;
      }
    }
    const float inv = 1.f / l;
    uint32_t w[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = E::pack2(acc[2 * k] * inv, acc[2 * k + 1] * inv);
    uint4* dst = reinterpret_cast<uint4*>(p.out + head * D + col);
    dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
    dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
    if (col == 0 && p.lse) p.lse[head] = (M + log2f(l)) * 0.6931471805599453f;
  }
}

template <int D, bool F16, bool SMALL>
__global__ void __launch_bounds__(THREADS, 1)
paged_attention_kernel(const __grid_constant__ PagedAttentionParams p, const __grid_constant__ CUtensorMap map_q,
                       const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                       const __grid_constant__ CUtensorMap map_o) {
  using C = ACfg<D, SMALL>;
  using E = Elem<F16>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                         ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
  uint64_t* q_full = bars;       // [tile]
  uint64_t* q_empty = bars + 2;  // [tile]
  uint64_t* k_full = bars + 4;
  uint64_t* k_empty = k_full + C::NK;
  uint64_t* v_full = k_empty + C::NK;
  uint64_t* v_empty = v_full + C::NV;
  uint64_t* s_full = v_empty + C::NV;  // [tile]
  uint64_t* p_full = s_full + 2;       // [tile]
  uint64_t* o_done = p_full + 2;       // [tile]
  uint64_t* v_land = o_done + 2;       // a sequence's last V tile has landed
  uint64_t* ml_full = v_land + 1;      // group B's m and l of a shared block are written
  uint64_t* ml_done = ml_full + 1;     // group A has read them and group B's accumulator
  uint64_t* part_full = ml_done + 1;   // SMALL: the partial result in slot 0, 1 is written
  uint64_t* drain = part_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::SLOT_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::FLAG_OFF);
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;  // (roles, hence addresses, the same in a warp)
  PagedCut* cut = static_cast<PagedCut*>(p.cuts) + blockIdx.x;

  if (warp == W_K && lane == 0) {
    tma_prefetch_map(&map_q);
    tma_prefetch_map(&map_k);
    tma_prefetch_map(&map_v);
  }
  pdl_wait();
  pdl_trigger();  // the next kernel may set itself up on SMs that are done here
  if (threadIdx.x == 0) cut->rows = 0;
  PagedRange range;
  if (!paged_range<THREADS>(p.m, p.status, p.num_ctas, UNITS_MIN, reinterpret_cast<int*>(smem + C::ML_OFF),
                            reinterpret_cast<PagedSeq*>(smem + C::SEQ_OFF), range,
                            [&](const PagedSeq& q) { return seq_units(p, q); }))
    return;  // uniform
  PagedWalk walk;
  walk.init(&p, range);
  if (!walk.ok) return;  // uniform: nothing but padding in this range

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NK; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 2);
    }
    for (int s = 0; s < C::NV; ++s) {
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 2);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&q_full[x], 1);
      mbar_init(&q_empty[x], 2);
      mbar_init(&s_full[x], 1);
      mbar_init(&p_full[x], SMALL ? 1 : 4);  // one arrival per softmax warp that works
      mbar_init(&o_done[x], 1);
    }
    mbar_init(v_land, 1);
    mbar_init(ml_full, SMALL ? 1 : 4);
    mbar_init(ml_done, SMALL ? 1 : 4);
    mbar_init(&part_full[0], 1);
    mbar_init(&part_full[1], 1);
    mbar_init(&drain[0], 1);
    mbar_init(&drain[1], 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == W_MMA) {
    tmem_alloc(tmem_slot, TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(*tmem_slot);
  const uint32_t sbase = uniform(smem_u32(smem));

  if (warp >= 8) {
  regs_dec<kRoleRegs>();
  // Whether every lane's wait succeeded (a timeout anywhere stops the warp).
#define KVGQA_WAIT(bar, parity) __all_sync(FULLMASK, mbar_wait_bounded((bar), (parity), abort_flag, p.status))
  if (warp == W_K) {
    // ------------------------------------------------------------ Q and K producer
    const uint64_t pol_q = l2_evict_first_policy();
    const uint64_t pol_kv = l2_evict_last_policy();  // re-read by the sequence's other blocks
    int it = 0, qn[2] = {0, 0};  // K tiles, and query tiles in each buffer, loaded so far
    // Query tile x of the block (0: A, 1: B) into buffer i.
    auto load_q = [&](int i, int x) -> bool {
      int& n = i == 0 ? qn[0] : qn[1];
      if (n >= 1 && !KVGQA_WAIT(&q_empty[i], (n - 1) & 1)) return false;
      if (lane == 0) {
        mbar_arrive_expect_tx(&q_full[i], (p.box_tokens << p.gp_shift) * D * 2);
        for (int sub = 0; sub < C::NSUB; ++sub)
          tma_load_4d(smem + C::Q_OFF + i * C::QTILE + sub * C::QSUB, &map_q, sub * 64, 0, walk.g,
                      walk.first + walk.tok0() + x * (BM >> p.gp_shift), &q_full[i], pol_q);
      }
      ++n;
      return true;
    };
    bool turns = false;  // the last tile went to one group
    TileBoxes t;
    for (; walk.ok; walk.advance()) {
      const bool fresh = walk.fresh(), dual = walk.dual();
      if (dual && turns) {
        // Both groups wait for every tile of this block, but of the last tiles
        // each knows its own only, and a barrier's parity does not tell a phase
        // from the one two before it: let the rings run dry first.
        bool dry = true;
        for (int u = max(it - C::NK, 0); u < it && dry; ++u) dry = KVGQA_WAIT(&k_empty[u % C::NK], (u / C::NK) & 1);
        for (int u = max(it - C::NV, 0); u < it && dry; ++u) dry = KVGQA_WAIT(&v_empty[u % C::NV], (u / C::NV) & 1);
        if (!dry) break;
      }
      turns = !dual;
      if (fresh) t.start(walk, lane);
      if (fresh && !load_q(dual ? 0 : walk.slot, 0)) break;
      const int s = it % C::NK;
      if (it >= C::NK && !KVGQA_WAIT(&k_empty[s], ((it / C::NK) - 1) & 1)) break;
      const int group = t.group(walk, lane);
      if (lane == 0) mbar_arrive_expect_tx(&k_full[s], t.n * t.rows * 128 * C::NSUB);
      __syncwarp();
      if (lane < t.n)
        tma_load_4d(smem + C::K_OFF + s * C::TILE + lane * t.rows * 128 * C::NSUB, &map_k, 0, 0, 0, group, &k_full[s],
                    pol_kv);
      t.fetch(walk, lane, walk.j + 1);
      ++it;
      if (fresh && dual && !load_q(1, 1)) break;
    }
    __syncwarp();
    if (*abort_flag) {  // let the copies in flight land
      volatile int none = 0;
      for (int x = 0; x < 2; ++x)
        if (qn[x] >= 1) mbar_wait_bounded(&q_full[x], (qn[x] - 1) & 1, &none, nullptr);
      for (int t = it - C::NK < 0 ? 0 : it - C::NK; t < it; ++t)
        mbar_wait_bounded(&k_full[t % C::NK], (t / C::NK) & 1, &none, nullptr);
    }
  } else if (warp == W_V) {
    // ------------------------------------------------------------ V producer
    const uint64_t pol_kv = l2_evict_last_policy();
    int it = 0, landed = 0;
    TileBoxes t;
    for (; walk.ok; walk.advance()) {
      const int s = it % C::NV;
      if (walk.fresh()) t.start(walk, lane);
      if (it >= C::NV && !KVGQA_WAIT(&v_empty[s], ((it / C::NV) - 1) & 1)) break;
      const int group = t.group(walk, lane);
      const int live = walk.kend - walk.j * BN;  // cells of this tile
      uint64_t* bar = live < BN ? v_land : &v_full[s];
      unsigned char* st = smem + C::V_OFF + s * C::TILE;
      if (lane == 0) mbar_arrive_expect_tx(bar, t.n * t.rows * 128 * C::NSUB);
      __syncwarp();
      if (lane < t.n) tma_load_4d(st + lane * t.rows * 128 * C::NSUB, &map_v, 0, 0, 0, group, bar, pol_kv);
      t.fetch(walk, lane, walk.j + 1);
      ++it;
      if (live < BN) {
        // the cells behind the last one weigh zero, and must not be NaN
        if (!KVGQA_WAIT(v_land, landed & 1)) break;
        ++landed;
        for (int i = live * 8 + lane; i < BN * 8; i += 32)
#pragma unroll
          for (int sub = 0; sub < C::NSUB; ++sub)
            *reinterpret_cast<uint4*>(st + (i >> 6) * C::Tile::GROUP + sub * 1024 + (i & 63) * 16) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&v_full[s]);
      }
    }
    __syncwarp();
    if (*abort_flag) {
      volatile int none = 0;
      mbar_wait_bounded(v_land, landed & 1, &none, nullptr);
      for (int t = it - C::NV < 0 ? 0 : it - C::NV; t < it; ++t)
        mbar_wait_bounded(&v_full[t % C::NV], (t / C::NV) & 1, &none, nullptr);
    }
  } else {
    // ------------------------------------------------------------ MMA issuers
    // Warp W_MMA + x issues the MMAs of group x: P.V of its last key tile, then
    // S of its next (in that order, since P lies over S).  Each issuer's waits
    // and bookkeeping pass while the tensor cores work on what the other has
    // issued: their queue is short, and one issuer for both groups left it empty
    // for a third of the time.  The whole warp runs the loop; one elected lane
    // issues the MMAs and their commits.  A stage is released by two arrivals:
    // one of each issuer, or two of the only one that uses it.
    constexpr uint32_t IDESC_QK = idesc_f16kind_f32(E::kMmaFormat, BM, BN, 0);
    constexpr uint32_t IDESC_PV = idesc_f16kind_f32(E::kMmaFormat, BM, D, 1);
    const uint32_t x = warp - W_MMA;
    const uint32_t s_tm = tmem + x * BN, o_tm = tmem + (2 + x) * BN;
    bool issued = false, ok = true;
    int n = 0;                // tiles of this group whose S has been issued
    int qn[2] = {0, 0};       // query tiles in each buffer so far
    int prev = -1;            // the tile whose P.V is next
    bool prev_first = false, prev_alone = false;
    // O_x (+)= P_x V of tile `prev`, by the elected lane
    auto issue_pv = [&]() {
      const uint32_t v_lo = smem_desc_lo(sbase + C::V_OFF + prev % C::NV * C::TILE, 1024);
#pragma unroll
      for (int ks = 0; ks < BN / 16; ++ks)
        umma_f16_ts_lo<C::Tile::GROUP>(o_tm, s_tm + ks * 8, v_lo + ks * (2 * C::Tile::GROUP >> 4), IDESC_PV, (ks > 0 || !prev_first) ? 1u : 0u);
    };
    auto release_v = [&]() {
      uint64_t* free = &v_empty[prev % C::NV];
      umma_commit(free);
      if (prev_alone) umma_commit(free);
    };
    auto wait_p = [&]() -> bool {
      return KVGQA_WAIT(&v_full[prev % C::NV], (prev / C::NV) & 1) && KVGQA_WAIT(&p_full[x], (n - 1) & 1);
    };
    auto finish_prev = [&]() -> bool {  // P.V of tile `prev`, if there is one
      if (prev < 0) return true;
      if (!wait_p()) return false;
      tc_fence_after();
      if (elect_one()) {
        issue_pv();
        umma_commit(&o_done[x]);
        release_v();
      }
      __syncwarp();
      prev = -1;
      return true;
    };
    for (; walk.ok && ok; walk.advance_segment()) {
      const bool dual = walk.dual();
      const int parts = walk.parts(), step = dual ? 1 : 2, from = dual || walk.group() == static_cast<int>(x) ? 0 : 1;
      const uint32_t i = dual ? x : uniform(walk.slot);  // the query buffer
      // A segment's last P.V waits for nothing of the next segment.
      ok = finish_prev();
      // Every issuer waits for every query tile and releases it, used or not,
      // so that neither misses a phase.
      for (uint32_t u = 0; u < 2 && ok; ++u) {
        if (!dual && u != i) continue;
        ok = KVGQA_WAIT(&q_full[u], (u == 0 ? qn[0] : qn[1]) & 1);
        if (u == 0) ++qn[0];
        else ++qn[1];
        if (ok && lane == 0 && (u != i || from >= parts)) mbar_arrive(&q_empty[u]);
      }
      if (!ok) break;
      for (int k = from; k < parts; k += step) {
        const int t = walk.ring + k, kn = t % C::NK;
        // Both groups at work on each tile: its K has long landed, so it is
        // waited for first and P.V and S go out without a gap.  The groups in
        // turn: the stream of K and V is the bound, and P.V does not wait for
        // a K tile that may still be on its way (its stage would be refilled
        // later for it).
        const bool together = dual && prev >= 0;
        if (!together && !(ok = finish_prev())) break;
        ok = KVGQA_WAIT(&k_full[kn], (t / C::NK) & 1) && (!together || wait_p());
        if (!ok) break;
        tc_fence_after();
        const uint32_t k_lo = smem_desc_lo(sbase + C::K_OFF + kn * C::TILE, 16);
        const uint32_t q_lo = smem_desc_lo(sbase + C::Q_OFF + i * C::QTILE, 16);
        if (elect_one()) {
          if (together) {
            issue_pv();
            umma_commit(&o_done[x]);  // (before the scores': a group that has seen those finds o_done a phase on)
          }
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t o = (ks % 4) * (32 >> 4);
            umma_f16_ss_lo<1024, C::Tile::GROUP>(s_tm, q_lo + (ks / 4) * (C::QSUB >> 4) + o,
                                                 k_lo + (ks / 4) * (1024 >> 4) + o, IDESC_QK, ks > 0);
          }
          umma_commit(&s_full[x]);
          umma_commit(&k_empty[kn]);
          if (!dual) umma_commit(&k_empty[kn]);
          if (together) release_v();
          if (k + step >= parts) umma_commit(&q_empty[i]);
        }
        __syncwarp();
        issued = true;
        prev = t;
        prev_first = k == from;
        prev_alone = !dual;
        ++n;
      }
    }
    if (ok) finish_prev();
    if (*abort_flag && issued) {
      // let every MMA issued so far finish before TMEM is released
      if (elect_one()) umma_commit(&drain[x]);
      __syncwarp();
      volatile int none = 0;
      mbar_wait_bounded(&drain[x], 0, &none, nullptr);
    }
  }
#undef KVGQA_WAIT
  } else {
    // ------------------------------------------------------------ softmax (warps 0-7)
    regs_inc<kSoftmaxRegs>();
    if (SMALL && (warp & 3) != 0) {
      // A small block's rows are one warp's (0 of its group).  Warp 1 counts the
      // CTA's partial results and merges a segment whose parts are complete: its
      // fence and its atomics would hold up the next segment elsewhere.
      if (warp == 1) {
        for (; walk.ok; walk.advance_segment()) {
          if (walk.whole()) continue;
          const bool starts = walk.vlo >= walk.v0;
          if (!__all_sync(FULLMASK, mbar_wait_bounded(&part_full[starts], 0, abort_flag, p.status))) break;
          __threadfence();
          __syncwarp();
          const int b0 = walk.vlo / range.w, b1 = walk.last_unit() / range.w;
          int* count = &static_cast<PagedCut*>(p.cuts)[b0].done;
          int before = 0;
          if (lane == 0) before = atomic_add_acq_rel_gpu(count, 1);
          if (__shfl_sync(FULLMASK, before, 0) == b1 - b0) {
            __syncwarp();  // (a shuffle orders no memory: lane 0's acquire becomes every lane's here)
            merge_small<D, F16>(p, walk.first, min(walk.ql << p.gp_shift, kSmallRows), walk.g, b0, b1);
            if (lane == 0) *count = 0;  // ready for the next call
          }
          __syncwarp();
        }
      }
    } else {
    const int x = warp >> 2;           // tile A or B
    const int r = threadIdx.x & 127;   // row of the tile == TMEM lane
    const int row_g = r & ((1 << p.gp_shift) - 1);   // head of the group
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + lane_base + x * BN;
    const uint32_t o_col = tmem + lane_base + (2 + x) * BN;
    const float c = p.scale_log2;
    const float ce = c > 0.f ? c : 1.f;
    float m_ref = -INFINITY, l = 0.f;
    float* ml = reinterpret_cast<float*>(smem + C::ML_OFF);
    int t = 0, t_other = 0;  // tiles of this group and of the other so far
    int n_shared = 0;        // shared parts so far
    for (; walk.ok; walk.advance_segment()) {
      const bool dual = walk.dual();
      // In a block without tile B both groups hold its 128 rows and take its
      // key tiles in turn.
      const int row0 = dual ? x * BM : 0;
      const int row_tok = (row0 + r) >> p.gp_shift;   // token of the row, within the block
      const int warp_tok = (row0 + (warp & 3) * 32) >> p.gp_shift;  // and of the warp's first row
      const bool live = walk.tok0() + warp_tok < walk.ql;  // the warp has rows of the sequence
      const int step = dual ? 1 : 2;
      const int seen = walk.off + walk.tok0();        // row r sees the cells up to seen + row_tok
      bool first = true;
      int j = walk.j_first + (dual || walk.group() == x ? 0 : 1);
      bool ok = true;
      for (; j < walk.j_end; j += step) {
      const int thr0 = seen - j * BN;  // column i of the tile is seen iff i <= thr
      const int thr = thr0 + row_tok;
      ok = __all_sync(FULLMASK, mbar_wait_bounded(&s_full[x], t & 1, abort_flag, p.status));
      if (!ok) break;
      if (live) {
      tc_fence_after();
      // Scores enter the softmax as s * ce with ce > 0 (a scale that is not
      // positive is folded into the scores first).
      uint32_t u[BN];
#pragma unroll
      for (int q = 0; q < BN / 32; ++q) tmem_ld32(s_col + q * 32, *reinterpret_cast<uint32_t(*)[32]>(u + q * 32));
      tmem_wait_ld();
      float* sv = reinterpret_cast<float*>(u);
      if (c <= 0.f) {
#pragma unroll
        for (int i = 0; i < BN; ++i) sv[i] *= c;
      }
      if (thr0 + warp_tok < BN - 1) {  // a tile that reaches past a row's cell
#pragma unroll
        for (int i = 0; i < BN; ++i) sv[i] = i <= thr ? sv[i] : -INFINITY;
      }
      float mx[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) mx[k] = fmaxf(sv[2 * k], sv[2 * k + 1]);
#pragma unroll
      for (int i = 16; i < BN; i += 16) {
#pragma unroll
        for (int k = 0; k < 8; ++k) mx[k] = fmax3(mx[k], sv[i + 2 * k], sv[i + 2 * k + 1]);
      }
      const float mraw = fmax3(fmax3(mx[0], mx[1], mx[2]), fmax3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7]));
      const float mt = mraw * ce;                    // tile maximum of the scaled scores
      const bool grow = first || mt > m_ref + 8.f;   // keep the old base unless it grew by 2^8
      float alpha = 1.f;
      if (grow) {
        alpha = first ? 0.f : ex2(m_ref - mt);
        m_ref = mt;
        l = first ? 0.f : l * alpha;  // (the last segment's row may have been padding, its sum anything)
      }
      // S_x of this tile being ready means the P.V of the previous tile is
      // complete, so O_x may be rescaled here without a further wait.
      if (__any_sync(FULLMASK, grow && !first)) {
#pragma unroll 1
        for (int q = 0; q < D / 32; ++q) {
          uint32_t w[32];
          tmem_ld32(o_col + q * 32, w);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * alpha);
          tmem_st32(o_col + q * 32, w);
        }
      }
      // A row that has seen no cell yet (the part of a cut segment may begin
      // in tiles that only later tokens see) keeps the base -inf; its weights
      // are 2^(-inf - 0) = 0.
      const float base = m_ref == -INFINITY ? 0.f : -m_ref;
      float2 ls = make_float2(0.f, 0.f);
      const float2 c2 = make_float2(ce, ce), nm2 = make_float2(base, base);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t w[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const int i0 = half * 64 + 2 * e;
          const float2 xx = ffma2(make_float2(sv[i0], sv[i0 + 1]), c2, nm2);
          const float2 pr = make_float2(ex2(xx.x), ex2(xx.y));
          ls = fadd2(ls, pr);
          w[e] = E::pack2(pr.x, pr.y);
        }
        tmem_st32(s_col + half * 32, w);
      }
      tmem_wait_st();
      l += ls.x + ls.y;
      }
      // Each warp arrives once: every lane's TMEM stores are complete and
      // fenced before the warp synchronises, then lane 0 arrives.
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[x]);
      ++t;
      first = false;
      }
      if (!ok) break;
      // ------------------------------------------------------ end of this part of the segment
      // A block without tile B whose part has two tiles or more is finished by
      // group A, which reads both accumulators (the lanes of tensor memory are
      // the same) once group B has left its m and l.
      const bool shared = !dual && walk.parts() > 1;
      t_other += dual ? walk.parts() : (walk.parts() + (walk.group() != x)) / 2;
      if (first) continue;  // no tile of this part was this group's
      float wa = 1.f, wb = 0.f;  // weights of the two accumulators
      if (shared) {
        const int ph = n_shared++ & 1;
        if (x == 1) {
          ml[r] = m_ref;
          ml[BM + r] = l;
          __syncwarp();
          if (lane == 0) mbar_arrive(ml_full);
          if (!__all_sync(FULLMASK, mbar_wait_bounded(ml_done, ph, abort_flag, p.status))) break;
          continue;
        }
        if (!__all_sync(FULLMASK, mbar_wait_bounded(ml_full, ph, abort_flag, p.status)) ||
            !__all_sync(FULLMASK, mbar_wait_bounded(&o_done[1], (t_other - 1) & 1, abort_flag, p.status)))
          break;
        const float mb = ml[r], lb = ml[BM + r];
        const float m = fmaxf(m_ref, mb);
        // (a group that saw none of the row's cells has m = -inf and weighs nothing)
        wa = m_ref == -INFINITY ? 0.f : ex2(m_ref - m);
        wb = mb == -INFINITY ? 0.f : ex2(mb - m);
        l = l * wa + lb * wb;
        m_ref = m;
      }
      const bool done = __all_sync(FULLMASK, mbar_wait_bounded(&o_done[x], (t - 1) & 1, abort_flag, p.status));
      tc_fence_after();
      const int tok = walk.tok0() + row_tok;
      const bool row_ok = tok < walk.ql && row_g < p.G;
      const uint32_t ob_col = tmem + lane_base + 3 * BN;
      // 32 values of the row from column q on: the merged accumulators
      auto read_o = [&](int q, uint32_t (&v)[32]) {
        tmem_ld32(o_col + q, v);
        if (shared) {
          uint32_t w[32];
          tmem_ld32(ob_col + q, w);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float o = wa > 0.f ? __uint_as_float(v[i]) * wa : 0.f;
            v[i] = __float_as_uint(wb > 0.f ? fmaf(__uint_as_float(w[i]), wb, o) : o);
          }
        } else {
          tmem_wait_ld();
        }
      };
      auto release_b = [&]() {  // group B's accumulator has been read
        if (shared) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(ml_done);
        }
      };
      if (done && live) {
        if (walk.whole()) {
          const float inv = 1.f / l;
          const size_t head = static_cast<size_t>(walk.first + tok) * p.H_q + walk.g * p.G + row_g;
          // This warp's 32 rows go out through shared memory and a TMA store
          // when all of its tokens belong to the sequence; else the rows that
          // do take direct stores.
          const bool via_tma = !SMALL && walk.tok0() + warp_tok + (32 >> p.gp_shift) <= walk.ql;
          unsigned char* stg = smem + C::STG_OFF + warp * C::STG;
          uint16_t* dst = p.out + head * D;
          if (row_ok && p.lse) p.lse[head] = (m_ref + log2f(l)) * 0.6931471805599453f;
#pragma unroll
          for (int sub = 0; sub < C::NSUB; ++sub) {  // 64 output values of the row at a time
            uint32_t w[32];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              uint32_t v[32];
              read_o(sub * 64 + half * 32, v);
#pragma unroll
              for (int k = 0; k < 16; ++k)
                w[half * 16 + k] = E::pack2(__uint_as_float(v[2 * k]) * inv, __uint_as_float(v[2 * k + 1]) * inv);
            }
            if (sub == C::NSUB - 1) release_b();
            if (via_tma) {
              if (lane == 0) bulk_wait_group_read<0>();  // the previous store has read the buffer
              __syncwarp();
#pragma unroll
              for (int k = 0; k < 8; ++k)  // 16-byte chunk k of row `lane` at its 128B-swizzled place
                *reinterpret_cast<uint4*>(stg + lane * 128 + ((k ^ (lane & 7)) << 4)) =
                    make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) {
                tma_store_4d(&map_o, stg, sub * 64, 0, walk.g, walk.first + walk.tok0() + warp_tok);
                bulk_commit_group();
              }
            } else if (row_ok) {
#pragma unroll
              for (int q16 = 0; q16 < 4; ++q16) {  // 16 values: a whole 32-byte sector
                uint16_t* o = dst + sub * 64 + q16 * 16;
                const uint32_t(&w8)[8] = *reinterpret_cast<const uint32_t(*)[8]>(w + 8 * q16);
                if (p.out_32b) {
                  stg256_stream(o, w8);
                } else {
                  *reinterpret_cast<uint4*>(o) = make_uint4(w8[0], w8[1], w8[2], w8[3]);
                  *reinterpret_cast<uint4*>(o + 8) = make_uint4(w8[4], w8[5], w8[6], w8[7]);
                }
              }
            }
          }
        } else {
          const bool starts = walk.vlo >= walk.v0;
          float* slot = p.partials + (static_cast<size_t>(blockIdx.x) * 2 + starts) * slot_floats(D);
          const int row = row0 + r;
          if (!SMALL && starts && row == 0) {
            cut->tok = walk.first + walk.tok0();
            cut->g = walk.g;
            cut->last = walk.last_unit() / range.w;
            cut->rows = min(ROWS, (walk.ql - walk.tok0()) << p.gp_shift);
          }
          if (row_ok) {
            slot[ROWS * D + row] = m_ref;
            slot[ROWS * D + ROWS + row] = l;
          }
#pragma unroll 1
          for (int q = 0; q < D / 32; ++q) {
            uint32_t v[32];
            read_o(q * 32, v);
            if (row_ok) {
#pragma unroll
              for (int k = 0; k < 8; ++k)
                *reinterpret_cast<uint4*>(slot + ((q * 8 + k) * ROWS + row) * 4) =
                    make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
            }
          }
          release_b();
          if constexpr (SMALL) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&part_full[starts]);
          }
        }
      }
      if (!done) break;
      if (!live) release_b();
    }
    }
  }

  if (warp < 8 && lane == 0) bulk_wait_group<0>();  // this warp's output stores are complete
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == W_MMA) tmem_dealloc(tmem, TMEM_COLS);
}

// ------------------------------------------------------------------ merge of cut segments
// Warp (b, y): 32 rows and 16 columns of the cut segment that starts in CTA b of
// the attention kernel, one row to a lane, so that a warp reads whole lines of
// each part.  A part whose maximum is -inf saw none of the row's cells and
// weighs nothing.
constexpr int kMergeWarps = 8;

template <int D, bool F16>
__global__ void __launch_bounds__(kMergeWarps * 32) paged_merge_kernel(const __grid_constant__ PagedAttentionParams p) {
  using E = Elem<F16>;
  pdl_wait();
  const int b0 = blockIdx.x, lane = threadIdx.x & 31;
  const int task = blockIdx.y * kMergeWarps + (threadIdx.x >> 5);
  const int row = task / (D / 16) * 32 + lane, col = task % (D / 16) * 16;
  const PagedCut cut = static_cast<const PagedCut*>(p.cuts)[b0];
  const int gi = row & ((1 << p.gp_shift) - 1);
  if (row >= cut.rows || gi >= p.G) return;
  auto part = [&](int b) { return p.partials + (static_cast<size_t>(b) * 2 + (b == b0)) * slot_floats(D); };
  float M = -INFINITY;
#pragma unroll 4
  for (int b = b0; b <= cut.last; ++b) M = fmaxf(M, part(b)[ROWS * D + row]);
  float l = 0.f, acc[16] = {};
#pragma unroll 2
  for (int b = b0; b <= cut.last; ++b) {
    const float* s = part(b);
    const float m = s[ROWS * D + row], lb = s[ROWS * D + ROWS + row];
    float4 o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = reinterpret_cast<const float4*>(s)[(col / 4 + k) * ROWS + row];
    if (m == -INFINITY) continue;
    const float w = exp2f(m - M);
    l += w * lb;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      acc[4 * k] += w * o[k].x;
      acc[4 * k + 1] += w * o[k].y;
      acc[4 * k + 2] += w * o[k].z;
      acc[4 * k + 3] += w * o[k].w;
    }
  }
  const float inv = 1.f / l;
  const size_t head = static_cast<size_t>(cut.tok + (row >> p.gp_shift)) * p.H_q + cut.g * p.G + gi;
  uint32_t w[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) w[k] = E::pack2(acc[2 * k] * inv, acc[2 * k + 1] * inv);
  uint4* dst = reinterpret_cast<uint4*>(p.out + head * D + col);
  dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
  dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
  if (col == 0 && p.lse) p.lse[head] = (M + log2f(l)) * 0.6931471805599453f;
}

// ------------------------------------------------------------------ host side
struct Maps {
  CUtensorMap q, k, v, o;
};

cudaError_t make_maps(const PagedAttentionParams& p, Maps* m) {
  auto enc = tma_encoder();
  if (!enc) return cudaErrorNotSupported;
  const CUtensorMapDataType type = p.f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const cuuint64_t D = p.D, G = p.G, Hkv = p.H_kv;
  const cuuint32_t es[4] = {1, 1, 1, 1};
  const cuuint32_t gp = 1u << p.gp_shift;
  for (int t = 0; t < 2; ++t) {  // q, and out in boxes of 32 rows
    const cuuint64_t dims[4] = {D, G, Hkv, static_cast<cuuint64_t>(p.m.N)};
    const cuuint64_t strides[3] = {D * 2, D * 2 * G, D * 2 * G * Hkv};
    const cuuint32_t box[4] = {64, gp, 1, t == 0 ? static_cast<cuuint32_t>(p.box_tokens) : 32 / gp};
    if (enc(t == 0 ? &m->q : &m->o, type, 4, t == 0 ? const_cast<uint16_t*>(p.q) : p.out, dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  if (paged_tile_map(enc, &m->k, type, p.k_cache, p.D, p.m.P, p.H_kv, p.m.page_shift) != CUDA_SUCCESS ||
      paged_tile_map(enc, &m->v, type, p.v_cache, p.D, p.m.P, p.H_kv, p.m.page_shift) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  return cudaSuccess;
}

template <int D, bool F16, bool SMALL>
cudaError_t launch_d(const PagedAttentionParams& p, const Maps& m, cudaStream_t stream) {
  using C = ACfg<D, SMALL>;
  static std::once_flag flags[64];
  static cudaError_t errs[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::call_once(flags[dev], [&] {
    const auto kernel = paged_attention_kernel<D, F16, SMALL>;
    errs[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    // setmaxnreg.inc is only satisfied if the launch hands out kLaunchRegs per thread.
    cudaFuncAttributes attr;
    if (errs[dev] == cudaSuccess) errs[dev] = cudaFuncGetAttributes(&attr, kernel);
    if (errs[dev] == cudaSuccess && attr.numRegs < kLaunchRegs) errs[dev] = cudaErrorInvalidConfiguration;
  });
  if (errs[dev] != cudaSuccess) return errs[dev];
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.num_ctas);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, paged_attention_kernel<D, F16, SMALL>, p, m.q, m.k, m.v, m.o);
  if (e != cudaSuccess || SMALL) return e;
  // As many rows as the segments' blocks can have.
  const int64_t rows = std::min<int64_t>(ROWS, static_cast<int64_t>(p.m.max_query_len) << p.gp_shift);
  const int64_t tasks = (rows + 31) / 32 * (D / 16);
  cfg.gridDim = dim3(p.num_ctas, static_cast<unsigned>((tasks + kMergeWarps - 1) / kMergeWarps));
  cfg.blockDim = dim3(kMergeWarps * 32);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, paged_merge_kernel<D, F16>, p);
}

bool is_small(const PagedAttentionParams& p) {
  return static_cast<int64_t>(p.m.max_query_len) << p.gp_shift <= kSmallRows;
}

template <int D>
cudaError_t launch_width(const PagedAttentionParams& p, const Maps& m, cudaStream_t stream) {
  if (is_small(p)) return p.f16 ? launch_d<D, true, true>(p, m, stream) : launch_d<D, false, true>(p, m, stream);
  return p.f16 ? launch_d<D, true, false>(p, m, stream) : launch_d<D, false, false>(p, m, stream);
}

}  // namespace

cudaError_t paged_attention_layout(int device, int D, PagedLayout* out) {
  static int sms[64];
  static std::once_flag flags[64];
  static cudaError_t errs[64];
  if (device < 0 || device >= 64) return cudaErrorInvalidDevice;
  std::call_once(flags[device], [&] {
    errs[device] = cudaDeviceGetAttribute(&sms[device], cudaDevAttrMultiProcessorCount, device);
  });
  if (errs[device] != cudaSuccess) return errs[device];
  out->num_ctas = sms[device];
  out->cut_bytes = (sms[device] * sizeof(PagedCut) + 255) / 256 * 256;
  out->partial_bytes = static_cast<size_t>(sms[device]) * 2 * slot_floats(D) * sizeof(float);
  return cudaSuccess;
}

cudaError_t launch_paged_attention(const PagedAttentionParams& params, cudaStream_t stream) {
  if (params.m.A == 0 || params.m.N == 0) return cudaSuccess;
  PagedAttentionParams p = params;
  p.out_32b = reinterpret_cast<uintptr_t>(p.out) % 32 == 0;
  p.gp_shift = 0;
  while ((1 << p.gp_shift) < p.G) ++p.gp_shift;
  // A query tile's box holds no more tokens than any sequence has (as a power
  // of two): a single token's tile is its own heads, and the rows behind them
  // are whatever the buffer held, which no other row sees.
  p.box_tokens = 1;
  while (p.box_tokens << p.gp_shift < BM && p.box_tokens < p.m.max_query_len) p.box_tokens *= 2;
  p.end_units = is_small(p) ? 2 : 4;
  Maps m;
  const cudaError_t e = make_maps(p, &m);
  if (e != cudaSuccess) return e;
  if (p.D == 128) return launch_width<128>(p, m, stream);
  if (p.D == 64) return launch_width<64>(p, m, stream);
  return cudaErrorInvalidValue;
}

}  // namespace kvgqa
