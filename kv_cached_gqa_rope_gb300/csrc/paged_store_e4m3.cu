// The store of the 8-bit paged cache: split-half RoPE with several position axes
// for the new queries and keys, fused with the store of keys and values as e4m3
// codes into the cells of a paged pool.
//
// The 16 cells 16 b .. 16 b + 15 of a page and KV head share a power of two as their
// scale.  With `bound` the largest magnitude that the block's new cells can have,
//   e = the least exponent byte with bound <= 448 * 2^(e - 127)
//   E = max(e, the block's exponent if it has older cells)
//   code = e4m3(value * 2^(127 - E)), to nearest even, of the FP32 value
// and where E has grown the older cells' codes are multiplied by 2^(E_old - E): exact
// but for codes that become subnormal, which are rounded.  A key's bound is the largest
// |x[i]| + |x[i + D/2]|, which no angle exceeds: it costs at most a bit of e4m3's range
// (none of its precision), depends on no position, and is known before the angles.
//
// Work.  A block's new cells have to be seen together, so a run (the new tokens of
// one block, 16 at most) is one CTA's.  A CTA looks at `chunk` packed tokens (1 or
// 16, see the launch) and takes the runs that begin there.  It evaluates the run's angles once
// for all heads into shared memory; a warp then takes a KV head's keys or values
// of the whole run (D / 16 lanes to a token, so that its reads and codes stay in
// registers between the bound and the rounding) and its share of the queries.  A
// single token's heads go side by side instead, D / 16 lanes each.  What a warp takes first
// is read before the angles, whose evaluation hides the latency.
// What bounds it, as measured (32 query, 8 KV heads of 128, BF16): a prefill of 16 x 1024
// tokens by memory, 72.4-73.6 us, 5.0-5.1 TB/s, three quarters of a copy's rate (the
// 16-bit store writes more and takes as long: here 16 reads lie between a block's bound and its
// first code); chunks with an image by latency, 9.6-9.7 us; 32 single tokens 3.9 us
// in a graph, 5.7 in calls, whose host side is longer.
// Measured and not kept, on the prefill: 3 CTAs an SM 86.7 us, 1 of 16 warps 87,
// 6 of 4 warps 91.6, 4 of 4 85; queries 8 heads a lane in flight instead of 4 88.8.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "e4m3.cuh"
#include "elem.cuh"
#include "paged.cuh"
#include "ptx.cuh"
#include "rope_math.cuh"

namespace kvgqa {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int kWarps = 8, kCtas = 2;  // of a CTA, and CTAs of an SM

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

// The 8 pairs (a[i], b[i]) turned, in FP32.
template <bool F16, int CH>
__device__ __forceinline__ void turn8(const uint4& a, const uint4& b, const float4* cs, float (&y1)[8], float (&y2)[8]) {
  using E = Elem<F16>;
  const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const float4 t = cs[w * CH];  // cos, sin of two neighbouring pairs
    const float2 c = make_float2(t.x, t.z), s = make_float2(t.y, t.w), ns = make_float2(-t.y, -t.w);
    const float2 x1 = E::pair_to_f2(aw[w]), x2 = E::pair_to_f2(bw[w]);
    const float2 u = ffma2(x1, c, fmul2(x2, ns)), v = ffma2(x2, c, fmul2(x1, s));
    y1[2 * w] = u.x;
    y1[2 * w + 1] = u.y;
    y2[2 * w] = v.x;
    y2[2 * w + 1] = v.y;
  }
}

template <bool F16>
__device__ __forceinline__ void unpack8(const uint4& a, float (&y)[8]) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = Elem<F16>::pair_to_f2(w[i]);
    y[2 * i] = v.x;
    y[2 * i + 1] = v.y;
  }
}

// Codes of 8 values times `inv`.
template <bool F16>
__device__ __forceinline__ uint2 code8(const float (&y)[8], float inv) {
  float z[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] = (F16 ? fminf(fmaxf(y[i], -kF16Most), kF16Most) : y[i]) * inv;
  return make_uint2(e4m3_pack4(z[0], z[1], z[2], z[3]), e4m3_pack4(z[4], z[5], z[6], z[7]));
}

// Four codes times f.
__device__ __forceinline__ uint32_t recode4(uint32_t x, float f) {
  const float2 a = __half22float2(e4m3_half2(x)), b = __half22float2(e4m3_half2(x >> 16));
  return e4m3_pack4(a.x * f, a.y * f, b.x * f, b.y * f);
}

template <int D, bool F16>
__global__ void __launch_bounds__(kWarps * 32, kCtas)
paged_rope_kv_store_e4m3_kernel(const __grid_constant__ PagedStoreParams p, int chunk, int trigger) {
  constexpr int HALF = D / 2;
  constexpr int CH = D / 16;           // lanes that share a head: 8 pairs each
  constexpr int HL = 32 / CH;          // heads a warp covers at a time
  constexpr int ROUNDS = kScaleCells / HL;
  // (cos, sin) of pair 8 c + 2 w + i of token t at [t][w][c][i]: the lanes that share
  // a head read neighbouring 16 bytes.
  __shared__ __align__(16) float2 cs_s[kScaleCells][HALF];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = lane % CH, sub = lane / CH;
  pdl_wait();
  if (trigger) pdl_trigger();
  const long long first_token = static_cast<long long>(blockIdx.x) * chunk;
  const int n0 = static_cast<int>(first_token), n1 = static_cast<int>(min(first_token + chunk, static_cast<long long>(p.m.N)));
  const int page = 1 << p.m.page_shift;

  int a = -1;
  PagedSeq seq{};
  bool busy = false;  // a run's angles may still be read
  for (int n = n0; n < n1;) {
    if (a < 0 || !seq.ok || n >= seq.first + seq.ql) {
      a = find_sequence(p.m, n);
      seq = paged_seq(p.m, a);
    }
    if (!seq.ok || n < seq.first || n >= seq.first + seq.ql) {  // a row of no sequence, or of one that is skipped
      if (!seq.ok && n >= seq.first && threadIdx.x == 0) atomicOr(p.status, KVGQA_FLAG_POSITION_RANGE);
      ++n;
      continue;
    }
    const int cell = seq.kl - seq.ql + (n - seq.first), older = cell & (kScaleCells - 1);
    const int len = min(kScaleCells - older, seq.first + seq.ql - n);
    if (older != 0 && n != seq.first) {  // the block's run began before
      n += len;
      continue;
    }
    const int pid = paged_page(p.m, a, cell);
    // The run's tokens with a negative position on an axis in use are skipped.
    bool neg = false;
    if ((lane & 15) < len) {
      for (int x = lane >> 4; x < p.axes; x += 2)
        neg = neg || ((p.axes_used >> x & 1) && p.positions[static_cast<size_t>(x) * p.m.N + n + (lane & 15)] < 0);
    }
    const unsigned ballot = __ballot_sync(FULL, neg);
    const unsigned bad = (ballot | ballot >> 16) & 0xffffu;
    const unsigned good = ((1u << len) - 1) & ~bad;
    if (threadIdx.x == 0) {
      if (bad) atomicOr(p.status, KVGQA_FLAG_POSITION_RANGE);
      if (good && pid < 0) atomicOr(p.status, KVGQA_FLAG_PAGE_RANGE);
    }
    if (!good || pid < 0) {  // uniform
      n += len;
      continue;
    }

    // What a warp takes first is read before the angles are known: a KV head's keys or
    // values of the run, or of a single token (a decode step) some of its heads, side
    // by side, D / 16 lanes to each.
    constexpr int FIRST = 2;
    static_assert(FIRST <= ROUNDS, "a single token's heads share the registers of a run's rounds");
    const int heads = p.H_q + 2 * p.H_kv;
    uint4 xa[ROUNDS], xb[ROUNDS];
    int fold[FIRST];
    auto head_source = [&](int h) {
      return h < p.H_q ? p.q + n * p.q_stride + h * D
             : h < p.H_q + p.H_kv ? p.k + n * p.k_stride + (h - p.H_q) * D : p.v + n * p.v_stride + (h - p.H_q - p.H_kv) * D;
    };
    auto scale_of = [&](int g, bool is_v) {  // of KV head g's block
      return (is_v ? p.v_scale : p.k_scale) + ((static_cast<size_t>(pid) * p.H_kv + g) << (p.m.page_shift - kScaleShift)) +
             ((cell & (page - 1)) >> kScaleShift);
    };
    auto codes_of = [&](int g, bool is_v) {  // of its first new cell
      return (is_v ? p.v_codes : p.k_codes) + ((static_cast<size_t>(pid) * p.H_kv + g) * page + (cell & (page - 1))) * D;
    };
    auto read_unit = [&](int unit) {
      const bool is_v = unit >= p.H_kv;
      const int g = is_v ? unit - p.H_kv : unit;
      const uint16_t* src = is_v ? p.v + n * p.v_stride + g * D : p.k + n * p.k_stride + g * D;
      const int64_t stride = is_v ? p.v_stride : p.k_stride;
#pragma unroll
      for (int b = 0; b < ROUNDS; ++b) {
        const int t = b * HL + sub;
        xa[b] = xb[b] = make_uint4(0, 0, 0, 0);
        if (good >> t & 1) {
          const uint16_t* s = src + t * stride;
          xa[b] = *reinterpret_cast<const uint4*>(s + c * 8);
          xb[b] = *reinterpret_cast<const uint4*>(s + HALF + c * 8);
        }
      }
    };
    if (len > 1) {
      if (warp < 2 * p.H_kv) read_unit(warp);
    } else {
#pragma unroll
      for (int b = 0; b < FIRST; ++b) {
        const int h = (warp + b * kWarps) * HL + sub;
        xa[b] = xb[b] = make_uint4(0, 0, 0, 0);
        fold[b] = 0;
        if (h >= heads) continue;
        xa[b] = *reinterpret_cast<const uint4*>(head_source(h) + c * 8);
        xb[b] = *reinterpret_cast<const uint4*>(head_source(h) + HALF + c * 8);
        const int kv = h - p.H_q;
        if (kv >= 0 && older) fold[b] = *scale_of(kv % p.H_kv, kv >= p.H_kv);
      }
    }

    if (busy) __syncthreads();
    busy = true;
    for (int i = threadIdx.x; i < len * HALF; i += kWarps * 32) {
      const int t = i / HALF, pair = i % HALF;
      const int pos = p.positions[static_cast<size_t>(p.axis[pair]) * p.m.N + n + t];
      cs_s[t][((pair >> 1 & 3) * CH + (pair >> 3)) * 2 + (pair & 1)] =
          rope_cos_sin_f32(pos, p.freqs.frac[pair], p.freqs.quad[pair]);
    }
    __syncthreads();

    if (len == 1) {
#pragma unroll 1
      for (int h0 = warp * HL; h0 < heads; h0 += kWarps * HL) {
        const int h = h0 + sub, kv = h - p.H_q;
        const bool is_q = kv < 0, is_v = kv >= p.H_kv, there = h < heads;
        const int g = is_v ? kv - p.H_kv : kv, b = h0 / (kWarps * HL);
        uint4 ya = b == 0 ? xa[0] : xa[1], yb = b == 0 ? xb[0] : xb[1];
        int old = b == 0 ? fold[0] : fold[1];
        if (b >= FIRST && there) {
          ya = *reinterpret_cast<const uint4*>(head_source(h) + c * 8);
          yb = *reinterpret_cast<const uint4*>(head_source(h) + HALF + c * 8);
          old = !is_q && older ? *scale_of(g, is_v) : 0;
        }
        float y1[8], y2[8], bound = 0.f;
        unpack8<F16>(ya, y1);
        unpack8<F16>(yb, y2);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          bound = fmaxf(bound, is_v ? fmaxf(fabsf(y1[i]), fabsf(y2[i])) : fabsf(y1[i]) + fabsf(y2[i]));
#pragma unroll
        for (int o = CH / 2; o; o >>= 1) bound = fmaxf(bound, __shfl_xor_sync(FULL, bound, o));
        if (!there) continue;
        if (!is_v) turn8<F16, CH>(ya, yb, reinterpret_cast<const float4*>(cs_s[0]) + c, y1, y2);
        if (is_q) {
          uint16_t* dst = p.q_out + (static_cast<size_t>(n) * p.H_q + h) * D;
          using E = Elem<F16>;
          *reinterpret_cast<uint4*>(dst + c * 8) =
              make_uint4(E::pack2(y1[0], y1[1]), E::pack2(y1[2], y1[3]), E::pack2(y1[4], y1[5]), E::pack2(y1[6], y1[7]));
          *reinterpret_cast<uint4*>(dst + HALF + c * 8) =
              make_uint4(E::pack2(y2[0], y2[1]), E::pack2(y2[2], y2[3]), E::pack2(y2[4], y2[5]), E::pack2(y2[6], y2[7]));
          continue;
        }
        const int e = max(old, e4m3_exponent(bound));
        uint8_t* codes = codes_of(g, is_v);
        if (c == 0 && (!older || e != old)) *scale_of(g, is_v) = static_cast<uint8_t>(e);
        if (older && e > old) {  // the older cells, coded again
          const int d = e - old;
          const float f = old == 0 || d > 126 ? 0.f : __uint_as_float(static_cast<uint32_t>(127 - d) << 23);
          for (int i = c * 16; i < older * D; i += CH * 16) {
            uint4* w = reinterpret_cast<uint4*>(codes - older * D + i);
            const uint4 x = *w;
            *w = make_uint4(recode4(x.x, f), recode4(x.y, f), recode4(x.z, f), recode4(x.w, f));
          }
        }
        const float inv = e == 0 ? 0.f : e4m3_inverse(e);
        *reinterpret_cast<uint2*>(codes + c * 8) = code8<F16>(y1, inv);
        *reinterpret_cast<uint2*>(codes + HALF + c * 8) = code8<F16>(y2, inv);
      }
      n += 1;
      continue;
    }

    // ---- keys and values
    for (int unit = warp; unit < 2 * p.H_kv; unit += kWarps) {
      const bool is_v = unit >= p.H_kv;
      const int g = is_v ? unit - p.H_kv : unit;
      if (unit != warp) read_unit(unit);
      uint8_t* scale = scale_of(g, is_v);
      uint8_t* codes = codes_of(g, is_v);
      int old = 0;
      if (older && lane == 0) old = *scale;
      old = __shfl_sync(FULL, old, 0);
      float bound = 0.f;
#pragma unroll
      for (int b = 0; b < ROUNDS; ++b) {
        float y1[8], y2[8];
        unpack8<F16>(xa[b], y1);
        unpack8<F16>(xb[b], y2);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          bound = fmaxf(bound, is_v ? fmaxf(fabsf(y1[i]), fabsf(y2[i])) : fabsf(y1[i]) + fabsf(y2[i]));
      }
      bound = __uint_as_float(__reduce_max_sync(FULL, __float_as_uint(bound)));  // (not negative: ordered as integers)
      const int e = max(old, e4m3_exponent(bound));
      if (lane == 0 && (!older || e != old)) *scale = static_cast<uint8_t>(e);
      if (older && e > old) {  // the older cells, coded again
        const int d = e - old;
        const float f = old == 0 || d > 126 ? 0.f : __uint_as_float(static_cast<uint32_t>(127 - d) << 23);
        for (int i = lane * 16; i < older * D; i += 512) {
          uint4* w = reinterpret_cast<uint4*>(codes - older * D + i);
          const uint4 x = *w;
          *w = make_uint4(recode4(x.x, f), recode4(x.y, f), recode4(x.z, f), recode4(x.w, f));
        }
      }
      const float inv = e == 0 ? 0.f : e4m3_inverse(e);
#pragma unroll
      for (int b = 0; b < ROUNDS; ++b) {
        const int t = b * HL + sub;
        if (!(good >> t & 1)) continue;
        float y1[8], y2[8];
        if (is_v) {
          unpack8<F16>(xa[b], y1);
          unpack8<F16>(xb[b], y2);
        } else {
          turn8<F16, CH>(xa[b], xb[b], reinterpret_cast<const float4*>(cs_s[t]) + c, y1, y2);
        }
        *reinterpret_cast<uint2*>(codes + t * D + c * 8) = code8<F16>(y1, inv);
        *reinterpret_cast<uint2*>(codes + t * D + HALF + c * 8) = code8<F16>(y2, inv);
      }
    }

    // ---- queries
    constexpr int QB = 4;  // heads in flight per lane
    const int items = len * p.H_q;
    for (int i0 = warp * HL + sub; i0 < items; i0 += kWarps * HL * QB) {
      uint4 qa[QB], qb[QB];
#pragma unroll
      for (int b = 0; b < QB; ++b) {
        const int i = i0 + b * kWarps * HL, t = i / p.H_q, h = i % p.H_q;
        if (i >= items || !(good >> t & 1)) continue;
        const uint16_t* s = p.q + (n + t) * p.q_stride + h * D;
        qa[b] = *reinterpret_cast<const uint4*>(s + c * 8);
        qb[b] = *reinterpret_cast<const uint4*>(s + HALF + c * 8);
      }
#pragma unroll
      for (int b = 0; b < QB; ++b) {
        const int i = i0 + b * kWarps * HL, t = i / p.H_q, h = i % p.H_q;
        if (i >= items || !(good >> t & 1)) continue;
        float y1[8], y2[8];
        turn8<F16, CH>(qa[b], qb[b], reinterpret_cast<const float4*>(cs_s[t]) + c, y1, y2);
        uint16_t* dst = p.q_out + (static_cast<size_t>(n + t) * p.H_q + h) * D;
        using E = Elem<F16>;
        *reinterpret_cast<uint4*>(dst + c * 8) =
            make_uint4(E::pack2(y1[0], y1[1]), E::pack2(y1[2], y1[3]), E::pack2(y1[4], y1[5]), E::pack2(y1[6], y1[7]));
        *reinterpret_cast<uint4*>(dst + HALF + c * 8) =
            make_uint4(E::pack2(y2[0], y2[1]), E::pack2(y2[2], y2[3]), E::pack2(y2[4], y2[5]), E::pack2(y2[6], y2[7]));
      }
    }
    n += len;
  }
}

// CTAs of the kernel that are resident on the device at a time.
template <int D, bool F16>
cudaError_t resident_ctas(int* ctas) {
  static std::once_flag flags[64];
  static cudaError_t errs[64];
  static int resident[64];
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::call_once(flags[dev], [&] {
    int sms = 0, per_sm = 0;
    errs[dev] = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (errs[dev] == cudaSuccess)
      errs[dev] = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, paged_rope_kv_store_e4m3_kernel<D, F16>,
                                                                kWarps * 32, 0);
    resident[dev] = sms * per_sm;
  });
  *ctas = resident[dev];
  return errs[dev];
}

template <int D, bool F16>
cudaError_t launch(const PagedStoreParams& p, cudaStream_t stream) {
  int ctas = 0;
  const cudaError_t e = resident_ctas<D, F16>(&ctas);
  if (e != cudaSuccess) return e;
  // A CTA for every token where they are resident together or sequences have 256 at most
  // in the mean, else one for every 16, whose runs go one after another: it costs most where
  // single tokens stand beside a prompt.  Measured, for every token and for every 16: 256 and 2048
  // sequences of one token 4.8 and 38, 27 and 41 us; 512 of 1-8 22 and 33; 63 single tokens
  // and one prompt of 1100 17 and 40, 22 and six of 40-512 18 and 35, 15 and one of 2048 20 and 40;
  // 32 of 24 15 and 21, of 64 20 and 19, of 128 32 and 27; 16 of 256 32 and 26; 5 of 301-1237 13.6
  // and 9.7; 16 of 1021-1024 97-100 and 72, 74 with 16 single tokens beside them; against
  // the rule 7 single tokens beside one prompt of 2048 19 and 30.
  const bool single = p.m.N <= ctas || p.m.N < 256ll * p.m.A;
  const int chunk = single ? 1 : kScaleCells;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((static_cast<long long>(p.m.N) + chunk - 1) / chunk));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // The next kernel may set itself up early only behind a short store: behind
  // a long one its CTAs would take SMs that this one's later CTAs need.
  return cudaLaunchKernelEx(&cfg, paged_rope_kv_store_e4m3_kernel<D, F16>, p, chunk, p.m.N <= ctas ? 1 : 0);
}

}  // namespace

cudaError_t launch_paged_rope_kv_store_e4m3(const PagedStoreParams& p, cudaStream_t stream) {
  if (p.m.N == 0 || p.m.A == 0) return cudaSuccess;
  if (p.D == 128) return p.f16 ? launch<128, true>(p, stream) : launch<128, false>(p, stream);
  if (p.D == 64) return p.f16 ? launch<64, true>(p, stream) : launch<64, false>(p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace kvgqa
