// Where a request's logical cache slot lives, for the kernels that take contiguous
// and paged caches alike, and the host checks of a paged cache's sizes.
#pragma once

#include "kd_common.cuh"

namespace kd {

// ------------------------------------------------------------------ slot -> cache row
// A request's logical slot s lives in cache row b * cap + s (contiguous caches) or in
// row page_table[b][s / P] * P + s % P of a shared page pool (paged caches: page size
// P > 1, the remedy for the page-size-1 fragmentation of "The Architectural Keystone",
// "Assumptions Embedded in the Design").
struct SlotMap {
  const int32_t* pt;          // [B][M] physical page ids, or nullptr for a contiguous cache
  int64_t cap;                // logical slots per request
  int64_t pages;              // pages in the pool (paged)
  int P, M;                   // page size, pages per request (paged)
  __device__ int64_t row(int b, int64_t s) const {
    return pt ? (int64_t)pt[(size_t)b * M + s / P] * P + s % P : (int64_t)b * cap + s;
  }
  // every page holding slots [s0, s1) is inside the pool (always true when contiguous)
  __device__ bool pages_ok(int b, int64_t s0, int64_t s1) const {
    if (!pt) return true;
    for (int64_t q = s0 / P; q <= (s1 - 1) / P; ++q) {
      const int32_t v = pt[(size_t)b * M + q];
      if (v < 0 || v >= pages) return false;
    }
    return true;
  }
};

// Sizes of a paged cache that the calls accept.
inline bool paged_ok(const int32_t* page_table, int page_size, int64_t pages_per_req, int64_t num_pages) {
  return page_table && page_size >= 1 && pages_per_req >= 1 && num_pages >= 1 &&
         num_pages * page_size <= (int64_t)INT32_MAX && pages_per_req * page_size <= (int64_t)INT32_MAX;
}

}  // namespace kd
