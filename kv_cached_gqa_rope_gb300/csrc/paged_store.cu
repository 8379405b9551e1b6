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
// written once (512 bytes per head at D = 128).  A warp takes some rounds of
// heads of a token (4 heads a round at D = 128) in a single round trip: all its
// loads are issued before the metadata and the angles are known.  It evaluates
// the D/2 angles two per lane; lane l then holds the cos/sin of its 8 pairs in
// registers and turns heads l / (D/16), + 32 / (D/16), ..., 32 bytes of each.
// V heads take the same path without the rotation.  What is left is the fixed
// cost of a token (its sequence, page and angles, a chain of loads), so warps
// take runs of consecutive tokens, which share sequence and page, where there
// are enough of them.  The angle is reduced exactly (integers) and the rest is
// FP32: a turned value is off by at most 2^-22 of its pair before it is rounded
// to the storage type.  16 x 1024 tokens with 32 + 8 + 8 heads of D = 128 take
// 72.9 us (5.5 TB/s read and written); one warp per token with all heads and
// the angles as double-float numbers took 94.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "elem.cuh"
#include "paged.cuh"
#include "ptx.cuh"
#include "rope_math.cuh"

namespace kvgqa {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int kWarps = 2;  // small CTAs: the registers of an SM hold more of them

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

// kBatch: heads in flight per lane.
template <int D, bool F16, int kBatch>
__global__ void __launch_bounds__(kWarps * 32)
paged_rope_kv_store_kernel(const __grid_constant__ PagedStoreParams p, int split, int chunk, int trigger) {
  constexpr int HALF = D / 2;
  constexpr int CH = D / 16;   // lanes that share a head: 8 pairs each
  constexpr int HL = 32 / CH;  // heads a warp covers at a time
  __shared__ __align__(16) float2 cs_s[kWarps][HALF];  // (cos, sin) of each pair, read two at a time
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  if (trigger) pdl_trigger();
  // This warp's share: heads part * kBatch * HL .. of the tokens n0 .. n1 - 1.
  const int w = blockIdx.x * kWarps + warp, part = w % split;
  const long long first_token = static_cast<long long>(w / split) * chunk;
  if (first_token >= p.m.N) return;
  const int n0 = static_cast<int>(first_token), n1 = min(n0 + chunk, p.m.N);
  const int heads = p.H_q + 2 * p.H_kv, rot_heads = p.H_q + p.H_kv;
  const int c = lane % CH, h0 = part * kBatch * HL + lane / CH;
  const int page = 1 << p.m.page_shift;
  const size_t head_step = static_cast<size_t>(page) * D;

  int a = -1, pid = -1, pid_cell = -1;  // the token's sequence; the page of cell pid_cell's page
  PagedSeq seq{};
  for (int n = n0; n < n1; ++n) {
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

    // The positions of this lane's pairs, and the token's cell.  Consecutive
    // tokens share their sequence and mostly their page.
    int pos[HALF / 32];
    bool pos_ok = true;
#pragma unroll
    for (int u = 0; u < HALF / 32; ++u) {
      pos[u] = p.positions[static_cast<size_t>(p.axis[lane + 32 * u]) * p.m.N + n];
      pos_ok = pos_ok && pos[u] >= 0;
    }
    if (a < 0 || !seq.ok || n >= seq.first + seq.ql) {
      a = find_sequence(p.m, n);
      seq = paged_seq(p.m, a);
      pid_cell = -1;
    }
    if (n < seq.first || (seq.ok && n >= seq.first + seq.ql)) continue;  // a row of no sequence
    pos_ok = __all_sync(FULL, pos_ok) && seq.ok;
    const int cell = seq.kl - seq.ql + (n - seq.first);
    if (seq.ok && (pid_cell < 0 || cell >> p.m.page_shift != pid_cell >> p.m.page_shift)) {
      pid = paged_page(p.m, a, cell);
      pid_cell = cell;
    }
    if (!pos_ok || pid < 0) {
      if (lane == 0) atomicOr(p.status, pos_ok ? KVGQA_FLAG_PAGE_RANGE : KVGQA_FLAG_POSITION_RANGE);
      continue;
    }
    const size_t cell_off = (static_cast<size_t>(pid) * p.H_kv * page + (cell & (page - 1))) * D;

    __syncwarp();  // (the last token's angles have been read)
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
}

// Warps of the kernel that are resident on the device at a time.
template <int D, bool F16, int kBatch>
cudaError_t resident_warps(int* warps) {
  static std::once_flag flags[64];
  static cudaError_t errs[64];
  static int resident[64];
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::call_once(flags[dev], [&] {
    int sms = 0, ctas = 0;
    errs[dev] = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (errs[dev] == cudaSuccess)
      errs[dev] = cudaOccupancyMaxActiveBlocksPerMultiprocessor(
          &ctas, paged_rope_kv_store_kernel<D, F16, kBatch>, kWarps * 32, 0);
    resident[dev] = sms * ctas * kWarps;
  });
  *warps = resident[dev];
  return errs[dev];
}

template <int D, bool F16, int kBatch>
cudaError_t launch_batch(const PagedStoreParams& p, int split, int chunk, cudaStream_t stream) {
  const long long warps = (static_cast<long long>(p.m.N) + chunk - 1) / chunk * split;
  if (warps > 0x7fffffffll) return cudaErrorInvalidValue;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((warps + kWarps - 1) / kWarps));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // The next kernel may set itself up early only behind a short store: behind
  // a long one its CTAs would take SMs that this one's later CTAs need.
  return cudaLaunchKernelEx(&cfg, paged_rope_kv_store_kernel<D, F16, kBatch>, p, split, chunk, chunk == 1 ? 1 : 0);
}

template <int D, bool F16>
cudaError_t launch(const PagedStoreParams& p, cudaStream_t stream) {
  constexpr int HL = 32 / (D / 16);
  const int heads = p.H_q + 2 * p.H_kv;
  auto split = [&](int batch) { return (heads + HL * batch - 1) / (HL * batch); };  // warps that share a token
  // With no more tokens than the GPU has warps for, each warp takes 4 rounds of
  // heads of one token (32 tokens: 3.4 us, with 6 rounds 3.7); beyond that 6
  // rounds, which the fixed cost of a token weighs less on, of a run of tokens
  // (16 x 1024 tokens: 72.9 us, with 4 rounds 79.0).
  int warps = 0;
  cudaError_t e = resident_warps<D, F16, 4>(&warps);
  if (e != cudaSuccess) return e;
  if (static_cast<long long>(p.m.N) * split(4) <= warps) return launch_batch<D, F16, 4>(p, split(4), 1, stream);
  e = resident_warps<D, F16, 6>(&warps);
  if (e != cudaSuccess) return e;
  const int shares = std::max(1, warps / split(6));  // runs of tokens in flight
  return launch_batch<D, F16, 6>(p, split(6), (p.m.N + shares - 1) / shares, stream);
}

}  // namespace

cudaError_t launch_paged_rope_kv_store(const PagedStoreParams& p, cudaStream_t stream) {
  if (p.m.N == 0 || p.m.A == 0) return cudaSuccess;
  if (p.D == 128) return p.f16 ? launch<128, true>(p, stream) : launch<128, false>(p, stream);
  if (p.D == 64) return p.f16 ? launch<64, true>(p, stream) : launch<64, false>(p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace kvgqa
