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
// written once (512 bytes per head at D = 128).  One warp takes kBatch rounds
// of heads of one token (16 heads at D = 128), a single round trip: all its
// loads are issued before the metadata and the angles are known.  It evaluates
// the D/2 angles two per lane; lane l then holds the cos/sin of its 8 pairs in
// registers and turns heads l / (D/16), + 32 / (D/16), ..., 32 bytes of each.
// V heads take the same path without the rotation.  A token's angles are
// evaluated once per warp that shares it, which costs less than the registers
// and the waiting of one warp that walks all heads: the prefill of 16 x 1024
// tokens with 32 + 8 + 8 heads took 94 us that way, with the angles as
// double-float numbers, and @@ us (@@ TB/s) like this.  The angle is reduced
// exactly (integers) and the rest is FP32: a turned value is off by at most
// 2^-22 of its pair before it is rounded to the storage type.
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

// x1 cos - x2 sin and x2 cos + x1 sin of two neighbouring pairs.
struct Turn2 {
  float2 c, s, ns;  // cos, sin, -sin
};
template <bool F16>
__device__ __forceinline__ void turn8(const uint4& a, const uint4& b, const Turn2 (&t)[4], uint4& ya, uint4& yb) {
  using E = Elem<F16>;
  const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
  uint32_t oa[4], ob[4];
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const float2 x1 = E::pair_to_f2(aw[w]), x2 = E::pair_to_f2(bw[w]);
    const float2 y1 = ffma2(x1, t[w].c, fmul2(x2, t[w].ns));
    const float2 y2 = ffma2(x2, t[w].c, fmul2(x1, t[w].s));
    oa[w] = E::pack2(y1.x, y1.y);
    ob[w] = E::pack2(y2.x, y2.y);
  }
  ya = make_uint4(oa[0], oa[1], oa[2], oa[3]);
  yb = make_uint4(ob[0], ob[1], ob[2], ob[3]);
}

template <int D, bool F16>
__global__ void __launch_bounds__(kWarps * 32)
paged_rope_kv_store_kernel(const __grid_constant__ PagedStoreParams p, int split, int trigger) {
  constexpr int HALF = D / 2;
  constexpr int CH = D / 16;   // lanes that share a head: 8 pairs each
  constexpr int HL = 32 / CH;  // heads a warp covers at a time
  __shared__ float2 cs_s[kWarps][HALF];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  if (trigger) pdl_trigger();
  const long long item = static_cast<long long>(blockIdx.x) * kWarps + warp;
  const int n = static_cast<int>(item / split), part = static_cast<int>(item % split);
  if (n >= p.m.N) return;
  const int heads = p.H_q + 2 * p.H_kv, rot_heads = p.H_q + p.H_kv;
  const int c = lane % CH, h0 = part * kBatch * HL + lane / CH;

  uint4 xa[kBatch], xb[kBatch];
#pragma unroll
  for (int b = 0; b < kBatch; ++b) {
    const int h = h0 + b * HL;
    if (h >= heads) continue;
    const uint16_t* s = h < p.H_q ? p.q + n * p.q_stride + h * D
                      : h < rot_heads ? p.k + n * p.k_stride + (h - p.H_q) * D
                                      : p.v + n * p.v_stride + (h - rot_heads) * D;
    xa[b] = *reinterpret_cast<const uint4*>(s + c * 8);
    xb[b] = *reinterpret_cast<const uint4*>(s + HALF + c * 8);
  }

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

#pragma unroll
  for (int u = 0; u < HALF / 32; ++u) {
    const int i = lane + 32 * u;
    cs_s[warp][i] = rope_cos_sin_f32(pos[u], p.freqs.frac[i], p.freqs.quad[i]);
  }
  __syncwarp();
  Turn2 t[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 v = *reinterpret_cast<const float4*>(&cs_s[warp][c * 8 + 2 * i]);
    t[i] = Turn2{make_float2(v.x, v.z), make_float2(v.y, v.w), make_float2(-v.y, -v.w)};
  }
#pragma unroll
  for (int b = 0; b < kBatch; ++b) {
    const int h = h0 + b * HL;
    if (h >= heads) continue;
    uint16_t* dst = h < p.H_q ? p.q_out + (static_cast<size_t>(n) * p.H_q + h) * D
                  : h < rot_heads ? p.k_cache + cell_off + (h - p.H_q) * head_step
                                  : p.v_cache + cell_off + (h - rot_heads) * head_step;
    uint4 ya = xa[b], yb = xb[b];
    if (h < rot_heads) turn8<F16>(xa[b], xb[b], t, ya, yb);
    *reinterpret_cast<uint4*>(dst + c * 8) = ya;
    *reinterpret_cast<uint4*>(dst + HALF + c * 8) = yb;
  }
}

template <int D, bool F16>
cudaError_t launch(const PagedStoreParams& p, cudaStream_t stream) {
  constexpr int HL = 32 / (D / 16);
  const int heads = p.H_q + 2 * p.H_kv;
  const int split = (heads + HL * kBatch - 1) / (HL * kBatch);  // warps that share a token
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
  return cudaLaunchKernelEx(&cfg, paged_rope_kv_store_kernel<D, F16>, p, split, grid <= 512 ? 1 : 0);
}

}  // namespace

cudaError_t launch_paged_rope_kv_store(const PagedStoreParams& p, cudaStream_t stream) {
  if (p.m.N == 0 || p.m.A == 0) return cudaSuccess;
  if (p.D == 128) return p.f16 ? launch<128, true>(p, stream) : launch<128, false>(p, stream);
  if (p.D == 64) return p.f16 ? launch<64, true>(p, stream) : launch<64, false>(p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace kvgqa
