// Tiles of 128 cells of a paged pool in shared memory, for the tensor cores.
// Internal to libkvgqa.
//
// The rows of a page lie one behind the other, so groups of 8 rows are a
// dimension of the pool that one box can take whole, both 64-column halves of a
// head of 128 with it:
//   [groups of 8 cells][D / 64 halves][8 cells][64 values, 128-byte swizzle].
// A page's part of a tile is then one TMA copy, whatever D is.  (The unit starts
// one copy in 66-90 clocks: 32 boxes of one half of 16 cells kept a producer
// warp 2100 clocks for 64 KB, 16 boxes of both halves 1000.)
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "paged.cuh"
#include "tcgen05.cuh"

namespace kvgqa {

template <int D>
struct PagedTile {
  static constexpr int CELLS = 128;
  static constexpr int HALVES = D / 64;
  static constexpr int GROUP = HALVES * 1024;        // bytes of 8 cells
  static constexpr int BYTES = CELLS / 8 * GROUP;
};

// The pool [P, H_kv, page, D] in groups of 8 rows; boxes of a page's cells, at
// most a tile's.
inline CUresult paged_tile_map(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap* map, CUtensorMapDataType type,
                               const uint16_t* pool, int D, int P, int H_kv, int page_shift) {
  const cuuint64_t d = D, page = 1ull << page_shift;
  const cuuint64_t dims[4] = {64, 8, d / 64, static_cast<cuuint64_t>(P) * H_kv * page / 8};
  const cuuint64_t strides[3] = {d * 2, 128, d * 16};
  const cuuint32_t box[4] = {64, 8, static_cast<cuuint32_t>(D / 64), static_cast<cuuint32_t>((page < 128 ? page : 128) / 8)};
  const cuuint32_t es[4] = {1, 1, 1, 1};
  return enc(map, type, 4, const_cast<uint16_t*>(pool), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

// A table's entry as it is, for a page looked at later (paged_tile_group): the
// read's latency passes meanwhile.
__device__ __forceinline__ int paged_entry(const PagedMeta& m, int a, int cell) {
  return m.block_table[static_cast<size_t>(a) * m.max_pages + (cell >> m.page_shift)];
}
// The group of 8 rows where `cell` (a multiple of 8) of KV head g lies in the
// pool; for an entry that is no page a place before the pool, from where a box
// reads zeros.
__device__ __forceinline__ int paged_tile_group(const PagedMeta& m, int entry, int H_kv, int g, int cell) {
  if (entry < 0 || entry >= m.P) return -PagedTile<64>::CELLS / 8;
  return ((entry * H_kv + g) << (m.page_shift - 3)) + ((cell & ((1 << m.page_shift) - 1)) >> 3);
}

}  // namespace kvgqa
