// The 8-bit cache: e4m3 codes, and the exponents of the scales that 16 cells of
// a KV head share.  Internal to libkvgqa.
//
// The exponent byte e stands for the scale 2^(e - 127), 0 for a scale of zero.
// Scales are powers of two, so that a code's value is exact in either 16-bit type
// (BF16 from 2^-126 on, IEEE binary16 in its range), a block's codes move to a
// larger scale exactly (down to e4m3's subnormals), and a product of codes is
// scaled by an addition to its exponent.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cudaTypedefs.h>

#include "paged.cuh"

namespace kvgqa {

constexpr int kScaleShift = 4;                 // 16 cells share a scale
constexpr int kScaleCells = 1 << kScaleShift;
// The largest value on e4m3's grid (times a power of two) that binary16 holds.
constexpr float kF16Most = 61440.f;

// The scale of an exponent byte.
__device__ __forceinline__ float e4m3_scale(int e) { return __uint_as_float(static_cast<uint32_t>(e) << 23); }
// Its reciprocal for e from 1 on (2^-127 is subnormal).
__device__ __forceinline__ float e4m3_inverse(int e) {
  return __uint_as_float(max(static_cast<uint32_t>(254 - e) << 23, 0x00400000u));
}
// 2^k for k up to 127: subnormal below 2^-126, 0 below 2^-149.
__device__ __forceinline__ float pow2(int k) {
  return __uint_as_float(k >= -126 ? static_cast<uint32_t>(k + 127) << 23 : k >= -149 ? 1u << (k + 149) : 0u);
}
// The least byte from 1 to 254 whose scale times 448 = 1.75 * 2^8 holds `bound`; 0 for 0.
__device__ __forceinline__ int e4m3_exponent(float bound) {
  const int e = static_cast<int>((__float_as_uint(bound) + 0x1fffffu) >> 23) - 8;
  return bound == 0.f ? 0 : min(max(e, 1), 254);
}

// Four values to four codes, rounded to nearest even, saturating at 448.
__device__ __forceinline__ uint32_t e4m3_pack4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}
// The values of two codes (in the low half of w), as binary16.
__device__ __forceinline__ __half2 e4m3_half2(uint32_t w) {
  const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w), __NV_E4M3);
  return *reinterpret_cast<const __half2*>(&r);
}

// The pool of codes [P, H_kv, page, D] in groups of 8 rows, in boxes of a page's
// cells, at most 128 of them: [cells][D bytes] in shared memory, swizzled over
// the row's bytes where the tensor cores read them.
inline CUresult e4m3_tile_map(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap* map, const uint8_t* pool, int D, int P,
                              int H_kv, int page_shift, bool swizzled) {
  const cuuint64_t d = D, page = 1ull << page_shift;
  const cuuint64_t dims[3] = {d, 8, static_cast<cuuint64_t>(P) * H_kv * page / 8};
  const cuuint64_t strides[2] = {d, d * 8};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(D), 8, static_cast<cuuint32_t>((page < 128 ? page : 128) / 8)};
  const cuuint32_t es[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(pool), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE,
             !swizzled ? CU_TENSOR_MAP_SWIZZLE_NONE : D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

// The exponent of the 16 cells from `cell` on of KV head g, where `entry` is
// the block table's for them; 0 for an entry that is no page.
__device__ __forceinline__ int e4m3_block_exponent(const PagedMeta& m, const uint8_t* scales, int entry, int H_kv, int g,
                                                   int cell) {
  if (entry < 0 || entry >= m.P) return 0;
  return scales[(static_cast<size_t>(entry * H_kv + g) << (m.page_shift - kScaleShift)) +
                ((cell & ((1 << m.page_shift) - 1)) >> kScaleShift)];
}

}  // namespace kvgqa
