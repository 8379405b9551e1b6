// The paged cache as the kernels see it: the packed new tokens of A sequences,
// their cells, and the block table that maps a sequence's cell to a page of
// the pool [P, H_kv, page, D].  Internal to libkvgqa.
#pragma once

#include <cstdint>

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
  s.ql = s.ok ? end - s.first : 0;
  return s;
}

// Page of cell `cell` of sequence a, or -1 where the table's entry is no page
// of the pool.
__device__ __forceinline__ int paged_page(const PagedMeta& m, int a, int cell) {
  const int pid = m.block_table[static_cast<size_t>(a) * m.max_pages + (cell >> m.page_shift)];
  return pid >= 0 && pid < m.P ? pid : -1;
}

}  // namespace kvgqa
