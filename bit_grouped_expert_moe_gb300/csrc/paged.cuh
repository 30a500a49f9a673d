// What the paged cache's kernels share (include/paged.h).
#pragma once

#include "common.cuh"
#include "paged.h"

namespace bgmoe {
namespace paged {

// Host checks shared by the entry points (paged_cache.cu).
bool shape_ok(const moe_paged_shape& s);
bool cache_ok(const moe_paged_cache* c);
inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

inline int page_shift(int page) { return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : page == 128 ? 7 : 8; }

}  // namespace paged
}  // namespace bgmoe
