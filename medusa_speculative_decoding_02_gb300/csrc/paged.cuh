// paged.cuh -- a cache in pages: where a slot lies.
//
// A pool of K (and one of V) is [n_pages][page][Hkv][dh].  Slot j of sequence b
// is row j % page of page table[b][j / page]; page is a power of two.
#pragma once

#include "common.cuh"

namespace medusa {

struct PageMap {
    const int32_t *table;  // [B][stride]
    int stride;            // pages a sequence may name
    int n_pages;
    int shift;             // log2(page)

    __device__ __forceinline__ int page_of(int b, int slot) const {
        return table[(size_t)b * stride + (slot >> shift)];
    }
    __device__ __forceinline__ bool good(int page) const {
        return (unsigned)page < (unsigned)n_pages;
    }
    // row of the pool that holds `slot`, which lies in `page`
    __device__ __forceinline__ size_t row(int page, int slot) const {
        return ((size_t)page << shift) + (slot & ((1 << shift) - 1));
    }
};

}  // namespace medusa
