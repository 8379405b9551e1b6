// The store of the paged cache: split-half RoPE with several position axes for
// the new queries and keys, fused with the store of keys and values into the
// cells of a paged pool.
//
// Pair i of a head, (x[i], x[i + D/2]), turns by the angle
// positions[axis_i][n] * theta^(-2i/D): text tokens carry the same position on
// every axis, a patch of an image or a video frame its time, row and column.
// The cell a token lands in (its sequence's next cell) and the position it is
// turned by are independent of each other.
//
// The kernel is bound by memory: every head of a token is read once and
// written once (512 bytes per head at D = 128), and the angles are D/2 per
// token whatever the heads.  One warp owns a token (or, with few tokens, a
// share of its heads, so that the loads of a decode step spread over the GPU
// and each warp waits for one round trip): it evaluates the D/2 angles two per
// lane, then lane l keeps the cos/sin of its 8 pairs in registers and streams
// heads l / (D/16), + 32 / (D/16), ..., 32 bytes in and out per head, with the
// first heads' loads issued before the metadata and the angles are known.
// V heads take the same path without the rotation.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "elem.cuh"
#include "paged.cuh"
#include "ptx.cuh"
#include "rope_math.cuh"

namespace kvgqa {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int kWarps = 8;
constexpr int kBatch = 4;  // heads in flight per lane

// The last sequence whose first row is at most n, by a 32-way search.
__device__ __forceinline__ int find_sequence(const PagedMeta& m, int n) {
  const int lane = threadIdx.x & 31;
  int lo = 0, len = m.A;
  while (len > 1) {
    const int step = (len + 31) / 32;
    const bool le = lane * step < len && m.query_starts[lo + lane * step] <= n;
    const int hit = max(__popc(__ballot_sync(FULL, le)) - 1, 0);
    lo += hit * step;
    len = min(step, len - hit * step);
  }
  return lo;
}

template <int D, bool F16>
__global__ void __launch_bounds__(kWarps * 32)
paged_rope_kv_store_kernel(const __grid_constant__ PagedStoreParams p, int split, int heads_per, int trigger) {
  constexpr int HALF = D / 2;
  constexpr int CH = D / 16;   // lanes that share a head: 8 pairs each
  constexpr int HL = 32 / CH;  // heads a warp covers at a time
  __shared__ CosSin cs_s[kWarps][HALF + HALF / 8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  if (trigger) pdl_trigger();
  const long long item = static_cast<long long>(blockIdx.x) * kWarps + warp;
  const int n = static_cast<int>(item / split), part = static_cast<int>(item % split);
  if (n >= p.m.N) return;
  const int heads = p.H_q + 2 * p.H_kv, rot_heads = p.H_q + p.H_kv;
  const int h_end = min(heads, (part + 1) * heads_per);
  const int c = lane % CH, hl = lane / CH;
  int h0 = part * heads_per + hl;

  auto src = [&](int h) -> const uint16_t* {
    if (h < p.H_q) return p.q + n * p.q_stride + h * D;
    if (h < rot_heads) return p.k + n * p.k_stride + (h - p.H_q) * D;
    return p.v + n * p.v_stride + (h - rot_heads) * D;
  };
  uint4 xa[kBatch], xb[kBatch];
  auto load = [&]() {
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int h = h0 + b * HL;
      if (h < h_end) {
        const uint16_t* s = src(h) + c * 8;
        xa[b] = *reinterpret_cast<const uint4*>(s);
        xb[b] = *reinterpret_cast<const uint4*>(s + HALF);
      }
    }
  };
  load();

  // The positions of this lane's pairs, and the token's cell.
  int pos[HALF / 32];
  bool pos_ok = true;
#pragma unroll
  for (int u = 0; u < HALF / 32; ++u) {
    pos[u] = p.positions[static_cast<size_t>(p.axis[lane + 32 * u]) * p.m.N + n];
    pos_ok = pos_ok && pos[u] >= 0;
  }
  const int a = find_sequence(p.m, n);
  const PagedSeq seq = paged_seq(p.m, a);
  const bool mine = n >= seq.first && (!seq.ok || n < seq.first + seq.ql);
  if (!mine) return;  // a row behind the last sequence
  pos_ok = __all_sync(FULL, pos_ok) && seq.ok;
  const int cell = seq.kl - seq.ql + (n - seq.first);
  const int pid = seq.ok ? paged_page(p.m, a, cell) : -1;
  if (!pos_ok || pid < 0) {
    if (lane == 0) atomicOr(p.status, pos_ok ? KVGQA_FLAG_PAGE_RANGE : KVGQA_FLAG_POSITION_RANGE);
    return;
  }
  const int page = 1 << p.m.page_shift;
  const size_t cell_off = (static_cast<size_t>(pid) * p.H_kv * page + (cell & (page - 1))) * D;
  const size_t head_step = static_cast<size_t>(page) * D;

  CosSin* cs = cs_s[warp];
#pragma unroll
  for (int u = 0; u < HALF / 32; ++u) {
    const int i = lane + 32 * u;
    cs[cs_slot(i)] = rope_cos_sin(pos[u], p.freqs.frac[i], p.freqs.quad[i]);
  }
  __syncwarp();
  CosSin mine_cs[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) mine_cs[i] = cs[cs_slot(c * 8) + i];

  for (;;) {
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int h = h0 + b * HL;
      if (h >= h_end) continue;
      uint16_t* dst = h < p.H_q ? p.q_out + (static_cast<size_t>(n) * p.H_q + h) * D
                    : h < rot_heads ? p.k_cache + cell_off + (h - p.H_q) * head_step
                                    : p.v_cache + cell_off + (h - rot_heads) * head_step;
      uint4 ya = xa[b], yb = xb[b];
      if (h < rot_heads) rotate8<F16>(xa[b], xb[b], mine_cs, ya, yb);
      *reinterpret_cast<uint4*>(dst + c * 8) = ya;
      *reinterpret_cast<uint4*>(dst + HALF + c * 8) = yb;
    }
    h0 += kBatch * HL;
    if (h0 - hl >= h_end) break;
    load();
  }
}

template <int D, bool F16>
cudaError_t launch(const PagedStoreParams& p, cudaStream_t stream) {
  constexpr int HL = 32 / (D / 16);
  const int heads = p.H_q + 2 * p.H_kv;
  // With fewer tokens than keep the GPU busy (two thousand warps), a token's
  // heads are shared out in whole rounds.
  const int rounds = (heads + HL * kBatch - 1) / (HL * kBatch);
  const int split = std::max(1, std::min(rounds, 2048 / std::max(1, p.m.N)));
  const int heads_per = (rounds + split - 1) / split * HL * kBatch;
  const long long items = static_cast<long long>(p.m.N) * split;
  const long long grid = (items + kWarps - 1) / kWarps;
  if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // The next kernel may set itself up early only behind a short store: behind
  // a long one its CTAs would take SMs that this one's later CTAs need.
  return cudaLaunchKernelEx(&cfg, paged_rope_kv_store_kernel<D, F16>, p, split, heads_per, grid <= 512 ? 1 : 0);
}

}  // namespace

cudaError_t launch_paged_rope_kv_store(const PagedStoreParams& p, cudaStream_t stream) {
  if (p.m.N == 0 || p.m.A == 0) return cudaSuccess;
  if (p.D == 128) return p.f16 ? launch<128, true>(p, stream) : launch<128, false>(p, stream);
  if (p.D == 64) return p.f16 ? launch<64, true>(p, stream) : launch<64, false>(p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace kvgqa
