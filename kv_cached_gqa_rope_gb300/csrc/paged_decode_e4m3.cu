// Attention over pools of 8-bit codes for blocks of at most 32 query rows (decode
// steps, a few tokens per sequence): codes go to the tensor cores as they lie in the
// pages, with no expansion on the way.
//
//   out[n, h] = sum_j softmax_j(scale * q[n, h] . k_j) v_j,  k_j, v_j = code * 2^(e - 127)
//
// Orientation.  The keys are the M side of both products, which few query rows
// would leave empty: per tile of 128 cells
//   S^T [128 keys, rows] = K Q^T          K from shared memory as it landed (K-major)
//   O^T [D, rows]       += V^T P^T        V as it landed (MN-major)
// on kind::f8f6f4.  Queries and weights are sums of 8-bit numbers, whose parts are
// further columns of the N side (N = rows x parts: the tile is read once for all):
//   queries  two (BF16) or three (binary16) e4m3 parts, each 2^5 of the one before:
//            a row times a power of two that brings its largest value to [2^7, 2^8),
//            q = q0 + 2^-5 q1 (+ 2^-10 q2): exact from 2^-14 (2^-16) of the largest on
//   weights  three (BF16) or four (binary16) e5m2 parts of the product with the value's
//            scale in binary16, each 2^3 of the one before: a relative error of binary16's
//            2^-11, with three parts 2^-9 more.  e5m2 is the upper half of binary16, so a part
//            is one addition, one mask and one subtraction for two rows.
// A key's scale multiplies its score, a value's its weight; both are one number to a
// thread.  A row has two bases: of its weights 2^x, whose sum is FP32, and of its
// products 2^(x + e) of weight and value scale, which become binary16 and parts: with one
// for the whole block, or against the largest scale, a large value that a row does not
// see, or that weighs nothing in it, would push its other products below binary16.
//
// Work.  Segments (sequence, KV head) of key tiles lie in one space of units, of
// which each CTA of the persistent grid takes an equal range (paged_walk.cuh); a segment cut
// by a boundary leaves FP32 partials, merged by the CTA that finishes last.
//   warps 0-7   softmax, one thread per key and half of the rows (a warpgroup each): FP32,
//               a row's bases follow its maxima when one of them grew by 2^6, which a
//               vote of the warpgroup finds out; only then is the maximum itself reduced and
//               the accumulator moved (tiles in turn instead, with a join of the two
//               at each segment's end: 32 sequences of up to 4095 cells 60 us where this took 46, the join 4 us);
//   warp 8      TMA of K, one box per page;
//   warp 9      the same for V; zeroes the cells behind a sequence's last one;
//   warp 10     tcgen05.mma of S^T, up to kBufs tiles ahead of the softmax; warp 14 of P.V (a
//               barrier costs its waiter about 140 clocks even when it is complete: with
//               one issuer for both they were the bound, 1500 clocks a tile);
//   warp 11     the rows of the queries in their parts, a segment ahead;
//   warp 12     merges the partials of a segment whose parts are complete;
//   warp 13     the scales of a tile to shared memory, some tiles ahead (their reads hang
//               on the block table's, which the copies need not wait for).
// What bounds it, as measured (8 KV heads of 128, BF16): long contexts by the stream of codes:
//   8 sequences of 65536 cells, 64 query heads, take 140 us, 6.3 TB/s, 92 % of the
//   rate of a copy (the 16-bit cache 263); shorter ones by that and by what does not shrink with
//   the cache, start, first tiles and 2-2.5 us for a segment's end: 32 sequences of up to
//   4095 cells, 32 query heads, 45.6-46 us, 2.9 TB/s (16 bits 57); 4 of up to 500 cells
//   7.6-7.9 us, all latency.  Where the stream is not the bound the softmax's instructions
//   are: two rows at a time in packed arithmetic, and a warp's maximum in one instruction, take
//   46 us there and 161 on 8 x 65536 cells with heads of 64 (16 bits 162), where single ones
//   took 49 and 205.  With 16 and 32 rows they are the longer part: 16 query heads to each of 4
//   KV heads, 8 x 65536 cells, 94 us (16 bits 151); 4 tokens on 32 x up to 4095 65 (62); 8 on
//   8 x 32768 183 (155).  FP16, with one part more of queries and weights, takes 156 us on 8 x
//   65536, 50 on 32 x 4095 and 237 for 8 tokens.  Measured on earlier forms and not kept: a
//   segment's end as 4 units, 343.7 us over five decode steps where 2 take 347.3, but 16 sequences of up to 8000 cells 41.1 where 39.2; MMAs issued by
//   single threads 72 and 251 us (operands that the compiler does not know to be uniform
//   cost 150 clocks an MMA); a wait for the room of the weights before the scores 175;
//   the scales at most two tiles ahead 49 and 158.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <mutex>

#include "e4m3.cuh"
#include "e4m3_tiles.cuh"
#include "elem.cuh"
#include "paged.cuh"
#include "paged_tiles.cuh"
#include "paged_walk.cuh"
#include "tcgen05.cuh"

namespace kvgqa {
namespace {

constexpr int THREADS = 15 * 32;
constexpr int W_K = 8, W_V = 9, W_S = 10, W_Q = 11, W_MERGE = 12, W_SCALE = 13, W_PV = 14;
constexpr int kBufs = 4;        // tiles whose scores, and whose weights, have room
constexpr int kTiles = 8;       // tiles whose scales are at hand
constexpr int kSegs = 8;        // segments whose rows' scales are at hand
constexpr float kWeightShift = 9.f; // products are times 2^9: at most 2^15 with their base's lag
constexpr float kLag = 6.f;
constexpr float kNone = -1e30f; // a row that has seen no cell: finite, so that no difference is NaN

struct __align__(16) KeyScales {
  float k[8];  // the scale of the keys' cells 16 i ..
  float v[8];  // the exponent byte of the values', -inf for a scale of zero
};

// NR: rows of a block, padded.
template <int D, bool F16, int NR>
struct DCfg {
  static constexpr int QP = F16 ? 3 : 2, PP = F16 ? 4 : 3;      // parts of queries and weights
  static constexpr int NS = (NR * QP + 15) / 16 * 16;           // columns of S^T
  static constexpr int NO = (NR * PP + 15) / 16 * 16;           // columns of O^T
  static constexpr int HR = NR / 2;                             // rows of a warpgroup
  static constexpr int TILE = BN * D;                           // bytes of a K or V tile
  static constexpr int STAGES = (NR == 32 ? 4 : NR == 16 ? 5 : 6) * 128 / D;  // of each
  static constexpr int K_OFF = 0;
  static constexpr int V_OFF = K_OFF + STAGES * TILE;
  static constexpr int QBUF = NS * 128, PBUF = NO * 128;
  static constexpr int Q_OFF = V_OFF + STAGES * TILE;           // two query buffers
  static constexpr int P_OFF = Q_OFF + 2 * QBUF;                // the weights of kBufs tiles
  static constexpr int TS_OFF = P_OFF + kBufs * PBUF;
  static constexpr int RQ_OFF = TS_OFF + kTiles * static_cast<int>(sizeof(KeyScales));  // the rows' scales of kSegs segments
  static constexpr int RED_OFF = RQ_OFF + kSegs * NR * 4;       // [warpgroup][4 warps]: maxima of its rows' scores and products, sums, flag
  static constexpr int RED = 4 * (3 * HR + 1) * 4;  // (a multiple of 16)
  static constexpr int SCR_OFF = RED_OFF + 2 * RED;             // the schedule's scratch
  static constexpr int SEQ_OFF = SCR_OFF + paged_scratch_bytes(THREADS);
  static constexpr int BAR_OFF = SEQ_OFF + kPagedSeqs * static_cast<int>(sizeof(PagedSeq));
  // k_full, k_empty, v_full, v_empty [STAGES], s_full, p_full, o_done [kBufs], q_full, q_empty, part_full [2],
  // scale_full, scale_empty [kTiles], v_land, drain [2]
  static constexpr int NBAR = 4 * STAGES + 3 * kBufs + 6 + 2 * kTiles + 3;
  static constexpr int SLOT_OFF = BAR_OFF + NBAR * 8;
  static constexpr int FLAG_OFF = SLOT_OFF + 8;
  static constexpr int SMEM = FLAG_OFF + 16 + 1024;             // + alignment slack
  static constexpr int O_COL = kBufs * NS;
  static constexpr int COLS = O_COL + NO;
  static constexpr int TMEM_COLS = COLS <= 64 ? 64 : COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
  static_assert(QBUF % 1024 == 0 && PBUF % 1024 == 0 && TILE % 1024 == 0, "swizzled tiles need 1024-byte alignment");
  static_assert(SMEM <= 232448 && COLS <= 512, "shared and tensor memory");
  static_assert(SEQ_OFF - SCR_OFF >= paged_scratch_bytes(THREADS), "the schedule's scratch");
};

// N columns of 32 lanes each.
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&v)[N]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  if constexpr (N == 4) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(taddr));
  } else if constexpr (N == 8) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]) : "r"(taddr));
  } else {
    tmem_ld16(taddr, *reinterpret_cast<uint32_t(*)[16]>(r));
  }
}
template <int N>
__device__ __forceinline__ void tmem_st(uint32_t taddr, const float (&v)[N]) {
  const uint32_t* r = reinterpret_cast<const uint32_t*>(v);
  if constexpr (N == 4) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
                 : "memory");
  } else if constexpr (N == 8) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
  } else {
    tmem_st16(taddr, *reinterpret_cast<const uint32_t(*)[16]>(r));
  }
}

// The largest of a warp's values; a NaN is none, unless all are.
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// Whether `p` holds for any thread of the 128 that meet at barrier `id`.
__device__ __forceinline__ bool vote_any(int id, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %2, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r) : "r"(id), "r"(static_cast<uint32_t>(p)) : "memory");
  return r != 0;
}

// One partial result: O [kSmallRows][D], then m and l [kSmallRows]; slot 2b + 1 of CTA b
// holds a segment that starts there, slot 2b one that started before.
constexpr size_t part_floats(int D) { return static_cast<size_t>(kSmallRows) * (D + 2); }

// One warp merges the parts b0 .. b1 of a block of `rows` rows (read past L1)
// and writes out and lse: a lane has a row's maximum and sum, then D / 32
// neighbouring columns of 8 rows at a time.
template <int D, bool F16>
__device__ __forceinline__ void merge_parts(const PagedAttentionParams& p, int tok0, int rows, int g, int b0, int b1) {
  using E = Elem<F16>;
  constexpr int C = D / 32, AT = 8;
  const int lane = threadIdx.x & 31;
  auto part = [&](int b) { return p.partials + (static_cast<size_t>(b) * 2 + (b == b0)) * part_floats(D); };
  float M = kNone, l = 0.f;  // of row `lane` (rows behind the last hold anything, and are not written)
#pragma unroll 4
  for (int b = b0; b <= b1; ++b) {
    const float m = __ldcg(part(b) + kSmallRows * D + lane), lb = __ldcg(part(b) + kSmallRows * (D + 1) + lane);
    const float to = fmaxf(M, m);
    // (a part that saw none of the row's cells weighs nothing)
    l = l * exp2f(M - to) + (m <= kNone ? 0.f : lb * exp2f(m - to));
    M = to;
  }
  const float inv = 1.f / l;
  for (int r0 = 0; r0 < rows; r0 += AT) {
    float acc[AT][C] = {};
#pragma unroll 2
    for (int b = b0; b <= b1; ++b) {
      const float* s = part(b);
      const float m = __ldcg(s + kSmallRows * D + lane);
      const float w = m <= kNone ? 0.f : exp2f(m - M) * inv;
      float o[AT][C];
#pragma unroll
      for (int i = 0; i < AT; ++i) {
        if constexpr (C == 4) *reinterpret_cast<float4*>(o[i]) = __ldcg(reinterpret_cast<const float4*>(s + (r0 + i) * D) + lane);
        else *reinterpret_cast<float2*>(o[i]) = __ldcg(reinterpret_cast<const float2*>(s + (r0 + i) * D) + lane);
      }
#pragma unroll
      for (int i = 0; i < AT; ++i) {
        const float wr = __shfl_sync(FULLMASK, w, r0 + i);
#pragma unroll
        for (int c = 0; c < C; ++c) acc[i][c] = wr > 0.f ? fmaf(wr, o[i][c], acc[i][c]) : acc[i][c];
      }
    }
#pragma unroll
    for (int i = 0; i < AT; ++i) {
      const int row = r0 + i, gi = row & ((1 << p.gp_shift) - 1);
      if (row >= rows || gi >= p.G) continue;
      const size_t head = static_cast<size_t>(tok0 + (row >> p.gp_shift)) * p.H_q + g * p.G + gi;
      uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + head * D) + lane * (C / 2);
#pragma unroll
      for (int c = 0; c < C / 2; ++c) dst[c] = E::pack2(acc[i][2 * c], acc[i][2 * c + 1]);
    }
  }
  const int gi = lane & ((1 << p.gp_shift) - 1);
  if (lane < rows && gi < p.G && p.lse)
    p.lse[static_cast<size_t>(tok0 + (lane >> p.gp_shift)) * p.H_q + g * p.G + gi] = (M + log2f(l)) * 0.6931471805599453f;
}

template <int D, bool F16, int NR>
__global__ void __launch_bounds__(THREADS, 1)
paged_decode_e4m3_kernel(const __grid_constant__ PagedAttentionParams p, const __grid_constant__ CUtensorMap map_k,
                         const __grid_constant__ CUtensorMap map_v) {
  using C = DCfg<D, F16, NR>;
  using E = Elem<F16>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                         ~static_cast<uintptr_t>(1023));
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
  uint64_t* k_empty = k_full + C::STAGES;
  uint64_t* v_full = k_empty + C::STAGES;
  uint64_t* v_empty = v_full + C::STAGES;
  uint64_t* s_full = v_empty + C::STAGES;  // [kBufs] S^T of a tile
  uint64_t* p_full = s_full + kBufs;       // [kBufs] its weights are written (and S^T read)
  uint64_t* o_done = p_full + kBufs;       // [kBufs] its P.V is complete
  uint64_t* q_full = o_done + kBufs;         // [2] the query buffer of segments of one parity
  uint64_t* q_empty = q_full + 2;
  uint64_t* part_full = q_empty + 2;       // [2] the partial result in slot 0, 1 is written
  uint64_t* scale_full = part_full + 2;    // [kTiles] a tile's scales are there,
  uint64_t* scale_empty = scale_full + kTiles;  // and have been used
  uint64_t* v_land = scale_empty + kTiles; // a sequence's last V tile has landed
  uint64_t* drain = v_land + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::SLOT_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::FLAG_OFF);
  KeyScales* scales = reinterpret_cast<KeyScales*>(smem + C::TS_OFF);
  float* q_scale = reinterpret_cast<float*>(smem + C::RQ_OFF);
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

  if (warp == W_K && lane == 0) {
    tma_prefetch_map(&map_k);
    tma_prefetch_map(&map_v);
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    for (int x = 0; x < kBufs; ++x) {
      mbar_init(&s_full[x], 1);
      mbar_init(&p_full[x], 8);  // one arrival per softmax warp
      mbar_init(&o_done[x], 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&drain[x], 1);
      mbar_init(&q_full[x], 1);
      mbar_init(&q_empty[x], 1);
      mbar_init(&part_full[x], 8);
    }
    for (int x = 0; x < kTiles; ++x) {
      mbar_init(&scale_full[x], 1);
      mbar_init(&scale_empty[x], 1);
    }
    mbar_init(v_land, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  pdl_wait();
  pdl_trigger();  // the next kernel may set itself up on SMs that are done here
  PagedRange range;
  if (!paged_range<THREADS>(p.m, p.status, p.num_ctas, UNITS_MIN, reinterpret_cast<int*>(smem + C::SCR_OFF),
                            reinterpret_cast<PagedSeq*>(smem + C::SEQ_OFF), range,
                            [&](const PagedSeq& q) { return seq_units(p, q); }))
    return;  // uniform
  PagedWalk walk;
  walk.init(&p, range);
  if (!walk.ok) return;  // uniform: nothing but padding in this range

  if (warp == W_S) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(*tmem_slot);
  const uint32_t sbase = uniform(smem_u32(smem));
#define KVGQA_WAIT(bar, parity) __all_sync(FULLMASK, mbar_wait_bounded((bar), (parity), abort_flag, p.status))

  if (warp == W_K) {
    // ------------------------------------------------------------ K
    const uint64_t pol = l2_evict_first_policy();
    TileBoxes t;
    int it = 0;
    for (; walk.ok; walk.advance(), ++it) {
      if (walk.fresh()) t.start(walk, lane);
      const int s = it % C::STAGES;
      if (it >= C::STAGES && !KVGQA_WAIT(&k_empty[s], ((it / C::STAGES) - 1) & 1)) break;
      const int group = t.group(walk, lane);
      if (lane == 0) mbar_arrive_expect_tx(&k_full[s], t.n * t.rows * D);
      __syncwarp();
      if (lane < t.n) tma_load_3d(smem + C::K_OFF + s * C::TILE + lane * t.rows * D, &map_k, 0, 0, group, &k_full[s], pol);
      t.fetch(walk, lane, walk.j + 1);
    }
    __syncwarp();
    if (*abort_flag) {  // let the copies in flight land
      volatile int none = 0;
      for (int u = it - C::STAGES < 0 ? 0 : it - C::STAGES; u < it; ++u)
        mbar_wait_bounded(&k_full[u % C::STAGES], (u / C::STAGES) & 1, &none, nullptr);
    }
  } else if (warp == W_SCALE) {
    // ------------------------------------------------------------ scales
    TileExponents ex;
    int t = 0;
    for (; walk.ok; walk.advance(), ++t) {
      if (walk.fresh()) ex.start(walk, lane);
      ex.advance(walk, lane);
      if (t >= kTiles && !KVGQA_WAIT(&scale_empty[t % kTiles], (t / kTiles - 1) & 1)) break;
      KeyScales& ks = scales[t % kTiles];
      if (lane < 8) ks.k[lane] = e4m3_scale(ex.e);
      else if (lane < 16) ks.v[lane - 8] = ex.e > 0 ? static_cast<float>(ex.e) : -INFINITY;
      __syncwarp();
      if (lane == 0) mbar_arrive(&scale_full[t % kTiles]);
    }
  } else if (warp == W_V) {
    // ------------------------------------------------------------ V
    const uint64_t pol = l2_evict_first_policy();
    TileBoxes t;
    int it = 0, landed = 0;
    for (; walk.ok; walk.advance()) {
      const int s = it % C::STAGES;
      if (walk.fresh()) t.start(walk, lane);
      if (it >= C::STAGES && !KVGQA_WAIT(&v_empty[s], ((it / C::STAGES) - 1) & 1)) break;
      const int group = t.group(walk, lane);
      const int live = walk.kend - walk.j * BN;  // cells of this tile
      uint64_t* bar = live < BN ? v_land : &v_full[s];
      unsigned char* st = smem + C::V_OFF + s * C::TILE;
      if (lane == 0) mbar_arrive_expect_tx(bar, t.n * t.rows * D);
      __syncwarp();
      if (lane < t.n) tma_load_3d(st + lane * t.rows * D, &map_v, 0, 0, group, bar, pol);
      t.fetch(walk, lane, walk.j + 1);
      ++it;
      if (live < BN) {
        // the cells behind the last one weigh zero, and must not be NaN (a row of the
        // tile is one of D bytes whatever the swizzle makes of it)
        if (!KVGQA_WAIT(v_land, landed & 1)) break;
        ++landed;
        for (int i = live * D / 16 + lane; i < C::TILE / 16; i += 32)
          *reinterpret_cast<uint4*>(st + i * 16) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&v_full[s]);
      }
    }
    __syncwarp();
    if (*abort_flag) {
      volatile int none = 0;
      mbar_wait_bounded(v_land, landed & 1, &none, nullptr);
      for (int u = it - C::STAGES < 0 ? 0 : it - C::STAGES; u < it; ++u)
        mbar_wait_bounded(&v_full[u % C::STAGES], (u / C::STAGES) & 1, &none, nullptr);
    }
  } else if (warp == W_S) {
    // ------------------------------------------------------------ S^T
    // Its columns are free when the weights of the tile kBufs before are written.  (The
    // operands of an MMA live in uniform registers: the whole warp runs the loop and one
    // lane issues; issued by a thread of its own each took 150 clocks.)
    constexpr uint32_t IDESC = idesc_e4m3_f32(BN, C::NS);
    constexpr uint32_t KHI = D == 128 ? desc_hi_sw128(1024) : desc_hi_sw64(512);
    int t = 0, seg = 0;
    for (; walk.ok; walk.advance(), ++t) {
      const uint32_t st = uniform(t % C::STAGES), b = uniform(t % kBufs), qb = uniform(seg & 1);
      const bool fresh = walk.fresh(), last = walk.j == walk.j_end - 1;
      if ((fresh && !KVGQA_WAIT(&q_full[qb], (seg >> 1) & 1)) || (t >= kBufs && !KVGQA_WAIT(&p_full[b], (t / kBufs - 1) & 1)) ||
          !KVGQA_WAIT(&scale_full[t % kTiles], (t / kTiles) & 1) || !KVGQA_WAIT(&k_full[st], (t / C::STAGES) & 1))
        break;
      tc_fence_after();
      const uint32_t k_lo = smem_desc_lo(sbase + C::K_OFF + st * C::TILE, 16);
      const uint32_t q_lo = smem_desc_lo(sbase + C::Q_OFF + qb * C::QBUF, 16);
      const uint32_t s_tm = tmem + b * C::NS;
      if (elect_one()) {
#pragma unroll
        for (int ks = 0; ks < D / 32; ++ks)
          umma_f8_ss_lo<KHI, desc_hi_sw128(1024)>(s_tm, k_lo + ks * (32 >> 4), q_lo + ks * (32 >> 4), IDESC, ks > 0);
        umma_commit(&s_full[b]);
        umma_commit(&k_empty[st]);
        if (last) umma_commit(&q_empty[qb]);
      }
      __syncwarp();
      if (last) ++seg;
    }
    if (*abort_flag && t > 0) {  // let every MMA issued so far finish before TMEM is released
      if (elect_one()) umma_commit(&drain[0]);
      __syncwarp();
      volatile int none = 0;
      mbar_wait_bounded(&drain[0], 0, &none, nullptr);
    }
  } else if (warp == W_PV) {
    // ------------------------------------------------------------ P.V
    constexpr uint32_t IDESC = idesc_e4m3_f32(BN, C::NO, 1, 1);
    constexpr uint32_t VHI = D == 128 ? desc_hi_sw128(1024) : desc_hi_sw64(512);
    int t = 0;
    for (; walk.ok; walk.advance(), ++t) {
      const uint32_t st = uniform(t % C::STAGES), b = uniform(t % kBufs);
      const uint32_t goes_on = uniform(!walk.fresh());
      if (!KVGQA_WAIT(&v_full[st], (t / C::STAGES) & 1) || !KVGQA_WAIT(&p_full[b], (t / kBufs) & 1)) break;
      tc_fence_after();
      // (at D = 64 the second half of M repeats the first)
      const uint32_t v_lo = smem_desc_lo(sbase + C::V_OFF + st * C::TILE, 0);
      const uint32_t p_lo = smem_desc_lo(sbase + C::P_OFF + b * C::PBUF, 16);
      const uint32_t o_tm = tmem + C::O_COL;
      if (elect_one()) {
#pragma unroll
        for (int ks = 0; ks < BN / 32; ++ks)
          umma_f8_ss_lo<VHI, desc_hi_sw128(1024)>(o_tm, v_lo + ks * (32 * D >> 4), p_lo + ks * (32 >> 4), IDESC, ks > 0 ? 1u : goes_on);
        umma_commit(&o_done[b]);
        umma_commit(&v_empty[st]);
        mbar_arrive(&scale_empty[t % kTiles]);  // (the softmax is through with the tile)
      }
      __syncwarp();
    }
    if (*abort_flag && t > 0) {
      if (elect_one()) umma_commit(&drain[1]);
      __syncwarp();
      volatile int none = 0;
      mbar_wait_bounded(&drain[1], 0, &none, nullptr);
    }
  } else if (warp == W_Q) {
    // ------------------------------------------------------------ queries in parts
    // (A buffer is free when the last scores from it are complete.  The rows' scales of
    // segment seg - kSegs have been read by then: the softmax is at most kBufs tiles behind
    // the scores, and every segment has a tile.)
    for (int seg = 0; walk.ok; walk.advance_segment(), ++seg) {
      if (seg >= 2 && !KVGQA_WAIT(&q_empty[seg & 1], ((seg >> 1) - 1) & 1)) break;
      const uint32_t buf = sbase + C::Q_OFF + (seg & 1) * C::QBUF;
      constexpr int V = D / 32;   // values of a lane
      constexpr int AT = 8;       // rows in flight
      const int rows = min(walk.ql << p.gp_shift, NR);
#pragma unroll 1
      for (int r0 = 0; r0 < NR; r0 += AT) {
        uint32_t raw[AT][V / 2];
#pragma unroll
        for (int i = 0; i < AT; ++i) {
          const int r = r0 + i, gi = r & ((1 << p.gp_shift) - 1);
#pragma unroll
          for (int k = 0; k < V / 2; ++k) raw[i][k] = 0;
          if (r < rows && gi < p.G) {
            const uint16_t* src = p.q + (static_cast<size_t>(walk.first + (r >> p.gp_shift)) * p.H_q + walk.g * p.G + gi) * D + lane * V;
            if constexpr (V == 4) {
              const uint2 w = *reinterpret_cast<const uint2*>(src);
              raw[i][0] = w.x;
              raw[i][1] = w.y;
            } else {
              raw[i][0] = *reinterpret_cast<const uint32_t*>(src);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < AT; ++i) {
          const int r = r0 + i;
          float v[4] = {};
          float m = 0.f;
#pragma unroll
          for (int k = 0; k < V / 2; ++k) {
            const float2 x = E::pair_to_f2(raw[i][k]);
            v[2 * k] = x.x;
            v[2 * k + 1] = x.y;
            m = fmax3(m, fabsf(x.x), fabsf(x.y));
          }
          const uint32_t top = __reduce_max_sync(FULLMASK, __float_as_uint(m));
          const int e = max(static_cast<int>(top >> 23), 16);  // (zeros, or tiny values: a factor of 2^118)
          const float f = __uint_as_float(static_cast<uint32_t>(127 + 134 - e) << 23);
          if (lane == 0) q_scale[seg % kSegs * NR + r] = __uint_as_float(static_cast<uint32_t>(e - 7) << 23);
#pragma unroll
          for (int k = 0; k < 4; ++k) v[k] *= f;
#pragma unroll
          for (int part = 0; part < C::QP; ++part) {
            const uint32_t x = e4m3_pack4(v[0], v[1], v[2], v[3]);
            const int row = part * NR + r;
            const uint32_t at = buf + row * 128 + ((((lane * V) >> 4) ^ (row & 7)) << 4) + ((lane * V) & 15);
            if constexpr (V == 4) asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(x) : "memory");
            else asm volatile("st.shared.b16 [%0], %1;" ::"r"(at), "h"(static_cast<uint16_t>(x)) : "memory");
            const float2 lo = __half22float2(e4m3_half2(x)), hi = __half22float2(e4m3_half2(x >> 16));
            v[0] = (v[0] - lo.x) * 32.f;
            v[1] = (v[1] - lo.y) * 32.f;
            v[2] = (v[2] - hi.x) * 32.f;
            v[3] = (v[3] - hi.y) * 32.f;
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[seg & 1]);
    }
  } else if (warp == W_MERGE) {
    // ------------------------------------------------------------ merge of cut segments
    for (; walk.ok; walk.advance_segment()) {
      if (walk.whole()) continue;
      const bool starts = walk.vlo >= walk.v0;
      if (!KVGQA_WAIT(&part_full[starts], 0)) break;
      __threadfence();
      __syncwarp();
      const int b0 = walk.vlo / range.w, b1 = walk.last_unit() / range.w;
      int* count = &static_cast<PagedCut*>(p.cuts)[b0].done;
      int before = 0;
      if (lane == 0) before = atomic_add_acq_rel_gpu(count, 1);
      if (__shfl_sync(FULLMASK, before, 0) == b1 - b0) {
        __syncwarp();  // (a shuffle orders no memory: lane 0's acquire becomes every lane's here)
        merge_parts<D, F16>(p, walk.first, min(walk.ql << p.gp_shift, NR), walk.g, b0, b1);
        if (lane == 0) *count = 0;  // ready for the next call
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ softmax (warps 0-7)
    constexpr int HR = C::HR;
    // Pairs of rows whose exponents stay in registers from the vote to the weights; more would
    // spill (8 tokens on 8 x 32768 cells, 16 rows here, 183 us, 203 with all kept; 16 query heads to
    // a KV head on 8 x 65536, 8 rows here, 94 us, 116 with none).
    constexpr int KEPT = HR / 2 < 4 ? HR / 2 : 4;
    const int wg = warp >> 2, quarter = warp & 3;
    const int key = quarter * 32 + lane;     // of the tile, == TMEM lane; of the result: the column d
    const int row0 = wg * HR;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t o_tm = tmem + lane_base + C::O_COL + row0;
    float* red = reinterpret_cast<float*>(smem + C::RED_OFF + wg * C::RED);  // maxima of the scores [4][HR]
    float* red_y = red + 4 * HR;                                            // and of the products' exponents [4][HR]
    float* sums = red_y + 4 * HR;                                           // [4][HR]
    int* red_ok = reinterpret_cast<int*>(sums + 4 * HR);                    // [4]
    const int bar_id = 1 + wg;
    // Of each row (two side by side): the base of its weights, negative, and their sum;
    // 2^kWeightShift over what the base of its products has more, in exponents (a whole number).
    float2 nm[HR / 2], l[HR / 2], nv[HR / 2];
    int t = 0;
    // A wait that gave up must not keep this warp from a barrier that the others of its
    // warpgroup come to: it goes on without effect until they leave together.
    bool alive = true, gone = false;
    for (int seg = 0; walk.ok; walk.advance_segment(), ++seg) {
      const int parts = walk.parts();
#pragma unroll
      for (int i = 0; i < HR / 2; ++i) {
        nm[i] = make_float2(-kNone, -kNone);
        l[i] = make_float2(0.f, 0.f);
        nv[i] = make_float2(kWeightShift, kWeightShift);
      }
      const float* rq = q_scale + seg % kSegs * NR + row0;
      for (int k = 0; k < parts; ++k, ++t) {
        const int j = walk.j_first + k, b = t % kBufs;
        alive = alive && KVGQA_WAIT(&s_full[b], (t / kBufs) & 1);
        float2 x[HR / 2];
        float ev;  // the value's exponent
        tc_fence_after();
        {
          float s[C::QP][HR];
#pragma unroll
          for (int part = 0; part < C::QP; ++part) tmem_ld<HR>(tmem + lane_base + b * C::NS + part * NR + row0, s[part]);
          const KeyScales& ks = scales[t % kTiles];
          const float kf = ks.k[key >> kScaleShift] * p.scale_log2;
          ev = ks.v[key >> kScaleShift];
          float2 q[HR / 2];
#pragma unroll
          for (int i = 0; i < HR / 2; i += 2) {
            const float4 w = *reinterpret_cast<const float4*>(rq + 2 * i);
            q[i] = make_float2(w.x, w.y);
            q[i + 1] = make_float2(w.z, w.w);
          }
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < HR / 2; ++i) {
            auto part = [&](int k) { return make_float2(s[k][2 * i], s[k][2 * i + 1]); };
            float2 d = ffma2(part(1), make_float2(0.03125f, 0.03125f), part(0));
            if (C::QP == 3) d = ffma2(part(C::QP - 1), make_float2(0.0009765625f, 0.0009765625f), d);
            x[i] = fmul2(d, fmul2(make_float2(kf, kf), q[i]));
          }
        }
        const int cell = j * BN + key;
        if ((j + 1) * BN > walk.off + 1) {   // a tile that reaches past a row's cell: row r sees those up to off + its token
#pragma unroll
          for (int r = 0; r < HR; ++r)
            if (cell > min(walk.off + ((row0 + r) >> p.gp_shift), walk.kend - 1)) (r & 1 ? x[r / 2].y : x[r / 2].x) = -INFINITY;
        }
        // The exponents of two rows' weights, and of their products with the value's scale.
        auto weight2 = [&](int i) { return fadd2(x[i], nm[i]); };
        auto product2 = [&](int i, float2 w) { return fadd2(w, fadd2(make_float2(ev, ev), nv[i])); };
        float2 w[KEPT], y[KEPT];
        float most_w = -INFINITY, most_y = -INFINITY;
#pragma unroll
        for (int i = 0; i < HR / 2; ++i) {
          const float2 wi = weight2(i), yi = product2(i, wi);
          if (i < KEPT) {
            w[i] = wi;
            y[i] = yi;
          }
          most_w = fmax3(most_w, wi.x, wi.y);
          most_y = fmax3(most_y, yi.x, yi.y);
        }
        if (vote_any(bar_id, !alive || most_w > kLag || most_y > kWeightShift + kLag)) {
          // The maxima of the tile, over the warpgroup.
#pragma unroll
          for (int r = 0; r < HR; ++r) {
            const float xr = r & 1 ? x[r / 2].y : x[r / 2].x;
            const float v = warp_max(xr), y = warp_max(xr + ev);
            if (lane == 0) {
              red[r * 4 + quarter] = v;
              red_y[r * 4 + quarter] = y;
            }
          }
          if (lane == 0) red_ok[quarter] = alive;
          // The accumulator is moved behind the P.V of its last tile.
          const bool move = k > 0;
          if (move) alive = alive && KVGQA_WAIT(&o_done[(t - 1) % kBufs], ((t - 1) / kBufs) & 1);
          named_bar_sync(bar_id, 128);
          if (!(red_ok[0] && red_ok[1] && red_ok[2] && red_ok[3])) {  // the same for all of them
            gone = true;
            break;
          }
          float alpha[HR];
#pragma unroll
          for (int r = 0; r < HR; ++r) {
            const float4 tx = *reinterpret_cast<const float4*>(red + 4 * r), ty = *reinterpret_cast<const float4*>(red_y + 4 * r);
            const float top = fmaxf(fmaxf(tx.x, tx.y), fmaxf(tx.z, tx.w)), top_y = fmaxf(fmaxf(ty.x, ty.y), fmaxf(ty.z, ty.w));
            // (A row that has seen no cell, or none with a scale, has a base near kNone, and
            // zeros so far.  The products' base falls by less than a binade where the
            // weights' alone grows, else it does not fall; as the latter is a maximum here, the
            // difference is 254 at most.)
            float& nmr = r & 1 ? nm[r / 2].y : nm[r / 2].x;
            float& nvr = r & 1 ? nv[r / 2].y : nv[r / 2].x;
            const float m = -nmr, vb = kWeightShift - nvr;
            const float to = fmaxf(m, top), by = floorf(fmaxf(m + vb, top_y) - to), a = m - to;
            alpha[r] = ex2(fminf(a + (vb - by), 1.f));
            (r & 1 ? l[r / 2].y : l[r / 2].x) *= ex2(a);
            nmr = -to;
            nvr = kWeightShift - by;
          }
#pragma unroll
          for (int i = 0; i < KEPT; ++i) {
            w[i] = weight2(i);
            y[i] = product2(i, w[i]);
          }
          if (move) {
            tc_fence_after();
#pragma unroll
            for (int part = 0; part < C::PP; ++part) {
              float o[HR];
              tmem_ld<HR>(o_tm + part * NR, o);
              tmem_wait_ld();
#pragma unroll
              for (int r = 0; r < HR; ++r) o[r] *= alpha[r];
              tmem_st<HR>(o_tm + part * NR, o);
            }
            tmem_wait_st();
          }
        }
        // The weights: exp2(x - m), and times the value's scale in their parts.
        const uint32_t pb = sbase + C::P_OFF + b * C::PBUF + (key & 15);
        if (t >= kBufs) alive = alive && KVGQA_WAIT(&o_done[b], (t / kBufs - 1) & 1);  // the buffer's last weights have been used
#pragma unroll
        for (int r = 0; r < HR; r += 2) {
          const int i = r / 2;
          const float2 wi = i < KEPT ? w[i < KEPT ? i : 0] : weight2(i), yi = i < KEPT ? y[i < KEPT ? i : 0] : product2(i, wi);
          l[i] = fadd2(l[i], make_float2(ex2(wi.x), ex2(wi.y)));
          __half2 h = __floats2half2_rn(ex2(yi.x), ex2(yi.y));
#pragma unroll
          for (int part = 0; part < C::PP; ++part) {
            const uint32_t c = (*reinterpret_cast<const uint32_t*>(&h) + 0x00800080u) & 0xff00ff00u;
            h = __hmul2(__hsub2(h, *reinterpret_cast<const __half2*>(&c)), __float2half2_rn(8.f));
            const int row = part * NR + row0 + r;
            asm volatile("st.shared.b8 [%0], %1;" ::"r"(pb + row * 128 + (((key >> 4) ^ (row & 7)) << 4)), "r"(c >> 8) : "memory");
            asm volatile("st.shared.b8 [%0], %1;" ::"r"(pb + (row + 1) * 128 + (((key >> 4) ^ ((row + 1) & 7)) << 4)), "r"(c >> 24)
                         : "memory");
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[b]);
      }
      if (gone) break;
      // ---------------------------------------------------------- end of this part of the segment
#pragma unroll
      for (int r = 0; r < HR; ++r) {
        float v = r & 1 ? l[r / 2].y : l[r / 2].x;
#pragma unroll
        for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(FULLMASK, v, o);
        if (lane == 0) sums[quarter * HR + r] = v;
      }
      alive = alive && KVGQA_WAIT(&o_done[(t - 1) % kBufs], ((t - 1) / kBufs) & 1);
      named_bar_sync(bar_id, 128);
      tc_fence_after();
      const int rows = min(walk.ql << p.gp_shift, NR);
      const bool whole = walk.whole(), starts = walk.vlo >= walk.v0;
      float* slot = p.partials + (static_cast<size_t>(blockIdx.x) * 2 + starts) * part_floats(D);
      float o[HR], sum[HR], m[HR];
#pragma unroll
      for (int r = 0; r < HR; ++r) o[r] = 0.f;
#pragma unroll
      for (int part = C::PP - 1; part >= 0; --part) {
        float v[HR];
        tmem_ld<HR>(o_tm + part * NR, v);
        tmem_wait_ld();
#pragma unroll
        for (int r = 0; r < HR; ++r) o[r] = fmaf(o[r], 0.125f, v[r]);
      }
#pragma unroll
      for (int r = 0; r < HR; ++r) {
        sum[r] = sums[r] + sums[HR + r] + sums[2 * HR + r] + sums[3 * HR + r];
        m[r] = -(r & 1 ? nm[r / 2].y : nm[r / 2].x);
        const float vb = kWeightShift - (r & 1 ? nv[r / 2].y : nv[r / 2].x);
        // (the products' base in two steps: by itself it may be below FP32's range)
        o[r] = o[r] * 0x1p-9f * pow2(static_cast<int>(fmaxf(vb, -1000.f)) - 127);
      }
      if (alive) {
#pragma unroll
        for (int r = 0; r < HR; ++r) {
          const int row = row0 + r, gi = row & ((1 << p.gp_shift) - 1);
          if (row >= rows || gi >= p.G) continue;
          if (whole) {
            const size_t head = static_cast<size_t>(walk.first + (row >> p.gp_shift)) * p.H_q + walk.g * p.G + gi;
            if (D == 128 || key < D) p.out[head * D + key] = E::from_f32(o[r] * __fdividef(1.f, sum[r]));
            if (key == 0 && p.lse) p.lse[head] = (m[r] + log2f(sum[r])) * 0.6931471805599453f;
          } else {
            if (D == 128 || key < D) slot[row * D + key] = o[r];
            if (key == 0) {
              slot[kSmallRows * D + row] = m[r];
              slot[kSmallRows * (D + 1) + row] = sum[r];
            }
          }
        }
      }
      if (!whole) {
        __syncwarp();
        if (lane == 0 && alive) mbar_arrive(&part_full[starts]);
      }
      tc_fence_before();
    }
  }
#undef KVGQA_WAIT

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == W_S) tmem_dealloc(tmem, C::TMEM_COLS);
}

// ------------------------------------------------------------------ host side
template <int D, bool F16, int NR>
cudaError_t launch(const PagedAttentionParams& p, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t stream) {
  using C = DCfg<D, F16, NR>;
  static std::once_flag flags[64];
  static cudaError_t errs[64];
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::call_once(flags[dev], [&] {
    errs[dev] = cudaFuncSetAttribute(paged_decode_e4m3_kernel<D, F16, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
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
  return cudaLaunchKernelEx(&cfg, paged_decode_e4m3_kernel<D, F16, NR>, p, k, v);
}

template <int D, bool F16>
cudaError_t launch_rows(const PagedAttentionParams& p, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(std::min(p.m.max_query_len, p.m.tokens_hi)) << p.gp_shift;
  if (rows <= 8) return launch<D, F16, 8>(p, k, v, stream);
  if (rows <= 16) return launch<D, F16, 16>(p, k, v, stream);
  return launch<D, F16, 32>(p, k, v, stream);
}

}  // namespace

cudaError_t launch_paged_attention_e4m3(const PagedAttentionParams& params, cudaStream_t stream) {
  PagedAttentionParams p = params;
  p.gp_shift = 0;
  while ((1 << p.gp_shift) < p.G) ++p.gp_shift;
  if (p.m.A == 0 || p.m.N == 0) return cudaSuccess;
  if (static_cast<int64_t>(p.m.max_query_len) << p.gp_shift > kSmallRows) {
    // Both kinds of sequences, as far as the host knows: chunks go to the kernel for
    // them, and those with as many tokens as the smallest form here holds (one at
    // least) follow.  (28 sequences of which 22 have one token: 151 us, 171 when all go
    // to the chunks' kernel; 64 of which 56 have one 161 and 254; without a small one the
    // launch in vain costs 5-8: 8 of 30-60 tokens 112 and 105.)
    const int most = std::max(8 >> p.gp_shift, 1);
    PagedAttentionParams chunks = params;
    chunks.m.tokens_lo = most + 1;
    const cudaError_t e = launch_paged_attention_e4m3_chunks(chunks, stream);
    if (e != cudaSuccess) return e;
    p.m.tokens_hi = most;
  }
  p.end_units = 2;
  auto enc = tma_encoder();
  if (!enc) return cudaErrorNotSupported;
  CUtensorMap k, v;
  if (e4m3_tile_map(enc, &k, p.k_codes, p.D, p.m.P, p.H_kv, p.m.page_shift, true) != CUDA_SUCCESS ||
      e4m3_tile_map(enc, &v, p.v_codes, p.D, p.m.P, p.H_kv, p.m.page_shift, true) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  if (p.D == 128) return p.f16 ? launch_rows<128, true>(p, k, v, stream) : launch_rows<128, false>(p, k, v, stream);
  if (p.D == 64) return p.f16 ? launch_rows<64, true>(p, k, v, stream) : launch_rows<64, false>(p, k, v, stream);
  return cudaErrorInvalidValue;
}

}  // namespace kvgqa
