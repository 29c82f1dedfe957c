// The 4-bit rows of an INT4 pool: where they lie, and the sizes every kernel on them shares.
#pragma once

#include "oscar_internal.cuh"

namespace oscar {

constexpr int kRow4 = kHeadDim / 2;                   // bytes of one row's codes

// log2 of the page size (16, 32 or 64): positions are split by shifts, not by divisions.
inline int page_shift(const oscar_layout_t &L) { return L.page_size == 16 ? 4 : L.page_size == 32 ? 5 : 6; }

// Row index of (page, kv head, slot) in the pool's arrays: a page holds one head's tokens together.
__device__ __forceinline__ size_t row4(int page, int n_kv, int h, int page_shift, int slot) {
    return (((size_t)page * n_kv + h) << page_shift) + slot;
}

}  // namespace oscar
