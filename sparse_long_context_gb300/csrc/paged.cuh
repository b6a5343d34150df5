// The paged K/V cache as its kernels see it, and its free pages.
//
// state: kPagedHead words, then a bit per page (1: free), then two words per sequence
// (the span of the append that is under way).  Head: word 0 the number of free
// pages, word 1 a word of the bits below which no page is free, word 2 whether the
// fork under way fails, word 3 the CTAs of the call under way that have arrived (0 between calls).
#pragma once

#include "common.cuh"
#include "launch.h"

namespace sls {

constexpr int kPagedHead = 16;
constexpr int kPagedMaxSeqs = 4096;  // sequences whose plans are kept in shared memory

__host__ __device__ inline int paged_words(int pages) { return (pages + 31) >> 5; }
__device__ __forceinline__ uint32_t* paged_bits(const Paged& c) { return reinterpret_cast<uint32_t*>(c.state + kPagedHead); }
__device__ __forceinline__ int2* paged_spans(const Paged& c) {  // an even number of words before them
  return reinterpret_cast<int2*>(c.state + kPagedHead + ((paged_words(c.pages) + 1) & ~1));
}
// Whether a table entry is a page of the pool.
__device__ __forceinline__ bool paged_page(int p, int pages) { return (unsigned)p < (unsigned)pages; }

}  // namespace sls
