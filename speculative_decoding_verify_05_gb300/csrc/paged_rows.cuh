// Packed ragged rows over a paged cache: which sequence a row belongs to, the bounds of a sequence, and loads and stores
// that bypass L1.  Args: the arguments of a kernel with cu_rows, ctx_len, B, M and max_pages.
#pragma once

#include "common.cuh"

#include <climits>

namespace spec {

// The last sequence with start(cu_rows[b], b) <= r, 32 candidates at a time by a whole warp; its lengths come with the
// last 32, so that they cost no load of their own after it.
struct Place {
  int b, c0, c1, ctx;                                   // b -1: r is before the first
};
template <class Args, class Start>
__device__ __forceinline__ Place place_of(int r, const Args& a, int lane, Start&& start) {
  int lo = 0, n = a.B;
  while (true) {
    const int step = (n + 31) >> 5, b = lo + lane * step;
    const bool in = b < lo + n, last = step == 1;
    int c0 = INT_MAX, c1 = 0, ctx = 0;
    if (in) {
      c0 = a.cu_rows[b];
      if (last) {
        c1 = a.cu_rows[b + 1];
        ctx = a.ctx_len[b];
      }
    }
    const unsigned votes = __ballot_sync(0xffffffffu, in && start(c0, b) <= r);
    if (votes == 0) return Place{-1, 0, 0, 0};          // (only before the first)
    const int k = 31 - __clz(votes);
    if (last)
      return Place{lo + k, __shfl_sync(0xffffffffu, c0, k), __shfl_sync(0xffffffffu, c1, k),
                   __shfl_sync(0xffffffffu, ctx, k)};
    n = min(step, n - k * step);
    lo += k * step;
  }
}

// The sequence of packed row r: the last that starts at or before it.
template <class Args>
__device__ __forceinline__ Place place_of(int r, const Args& a, int lane) {
  return place_of(r, a, lane, [](int c0, int) { return c0; });
}

// 16 bytes past L1, which has no use for them.
__device__ __forceinline__ uint4 ld_past_l1(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ void st_past_l1(uint16_t* p, const uint4& v) {
  asm volatile("st.global.L1::no_allocate.v4.b32 [%0], {%1,%2,%3,%4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

// Whether a sequence is outside the M rows or past its table's keys (its length and pages count only if it has rows).
template <class Args>
__device__ __forceinline__ bool out_of_bounds(int c0, int c1, int ctx, const Args& a) {
  constexpr int PAGE = 128;
  return c0 < 0 || c1 < c0 || c1 > a.M ||
         (c1 > c0 && (ctx < 0 || (long long)ctx + (c1 - c0) > (long long)a.max_pages * PAGE));
}

}  // namespace spec
