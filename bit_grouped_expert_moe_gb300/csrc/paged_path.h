// The rule for one entry of a sequence's path of accepted drafts (moe_paged_keep,
// include/paged.h). Plain C++, so that a test without a GPU can go through it.
#pragma once

#ifdef __CUDACC__
#define BGMOE_HD __host__ __device__ __forceinline__
#else
#define BGMOE_HD inline
#endif

namespace bgmoe {
namespace paged {

// Whether entry k, `from`, may be looked up in the page table, given the entry
// before it (-1 before the first) and 0 <= start <= limit. Each entry is judged on
// its own, by a thread that does not know of the others' errors, so the answer has
// to bound both of the entry's positions, start + from and start + k, by itself:
// entries of a path that increases from 0 or more have from >= k.
BGMOE_HD bool path_entry_ok(int from, int before, int k, int start, long long limit) {
  return from > before && from >= k && start + (long long)from < limit;
}

}  // namespace paged
}  // namespace bgmoe
