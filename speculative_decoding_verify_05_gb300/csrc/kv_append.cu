// Prompt side of the paged cache, the two kernels before the attention of a chunk: the rotation table
// of positions with several axes, and the append of a chunk's keys and values to their pages with the
// rotation applied on the way.
#include "common.cuh"
#include "internal.h"

namespace spec {
namespace {

constexpr int D = 128;
constexpr int PAGE = 128;

// (cos, sin) of x turns, x = u / 2^64.  The position times the frequency is formed modulo one turn in 64-bit
// integers (wrap-around is the reduction, exact for any 32-bit position), the nearest quarter turn
// is split off, and what is left, at most an eighth of a turn, is exact to 2^-33 turns before its one
// rounding to fp32.  No fp64 instruction: the chip has few of them.
__device__ __forceinline__ float2 cos_sin_turns(unsigned long long u) {
  const unsigned hi = (unsigned)(u >> 32);
  const unsigned quarter = (hi + (1u << 29)) >> 30;                 // 0..4, 4 = 0
  const int rem = (int)(hi - (quarter << 30));                      // [-2^29, 2^29)
  float s, c;
  sincospif((float)rem * 0x1p-31f, &s, &c);                         // 2 pi rem / 2^32 = pi (rem / 2^31)
  switch (quarter & 3u) {
    case 0: return make_float2(c, s);
    case 1: return make_float2(-s, c);
    case 2: return make_float2(-c, -s);
    default: return make_float2(s, -c);
  }
}

// One thread per table entry.
__global__ void __launch_bounds__(256)
rope_table_axes_kernel(const int32_t* __restrict__ pos, int ldpos, int M, int half, const __grid_constant__ RopeAxes f,
                       float2* __restrict__ cs) {
  pdl_wait();
  pdl_trigger();
  const long long total = (long long)M * half;
  for (long long idx = blockIdx.x * 256ll + threadIdx.x; idx < total; idx += gridDim.x * 256ll) {
    const int r = (int)(idx / half), i = (int)(idx - (long long)r * half);
    const int p = pos[(size_t)f.axis[i] * ldpos + r];
    cs[idx] = cos_sin_turns((unsigned long long)(long long)p * f.turn[i]);
  }
}

// One CTA per row; a thread moves one 8-element pair of chunks (i, i + 64) of a head at a time.
__global__ void __launch_bounds__(128) kv_append_kernel(const KvAppendArgs a) {
  pdl_wait();
  pdl_trigger();
  const int r = blockIdx.x;
  int lo = 0, hi = a.B - 1;
  while (lo < hi) {                     // the last sequence with cu_rows[b] <= r
    const int mid = (lo + hi + 1) >> 1;
    if (a.cu_rows[mid] <= r) lo = mid; else hi = mid - 1;
  }
  const int c0 = a.cu_rows[lo], c1 = a.cu_rows[lo + 1], ctx = a.ctx_len[lo];
  if (r < c0 || r >= c1) return;        // padding
  if (c0 < 0 || c1 > a.M || ctx < 0 || (long long)ctx + (c1 - c0) > (long long)a.max_pages * PAGE) {
    if (threadIdx.x == 0) set_status(a.status, 0x6F1u);
    return;
  }
  const int p = ctx + (r - c0);
  const int page = a.block_table[(size_t)lo * a.max_pages + p / PAGE];
  const bool bad = page < 0 || page >= a.num_pages;
  if (bad && threadIdx.x == 0) set_status(a.status, 0x6F2u);
  for (int u = threadIdx.x; u < (a.Hq + 2 * a.Hkv) * 8; u += 128) {
    const int hd = u >> 3, i0 = (u & 7) * 8;
    const uint16_t* src;
    uint16_t* dst;
    bool turn = a.cs != nullptr;
    if (hd < a.Hq) {
      src = a.Q + (size_t)r * a.ldq + (size_t)hd * D;
      dst = a.Qrot + (size_t)r * a.ldqr + (size_t)hd * D;
    } else {
      if (bad) continue;
      const bool is_v = hd >= a.Hq + a.Hkv;
      const int g = hd - a.Hq - (is_v ? a.Hkv : 0);
      turn = turn && !is_v;
      src = (is_v ? a.Vnew : a.Knew) + (size_t)r * a.ldkv + (size_t)g * D;
      dst = (is_v ? a.Vpool : a.Kpool) + (((size_t)g * a.num_pages + page) * PAGE + p % PAGE) * D;
    }
    uint4 x = *reinterpret_cast<const uint4*>(src + i0), y = *reinterpret_cast<const uint4*>(src + 64 + i0);
    if (turn) {
      uint32_t* xa = reinterpret_cast<uint32_t*>(&x);
      uint32_t* ya = reinterpret_cast<uint32_t*>(&y);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 t0 = a.cs[(size_t)r * 64 + i0 + 2 * e], t1 = a.cs[(size_t)r * 64 + i0 + 2 * e + 1];
        const float a0 = bf16lo(xa[e]), a1 = bf16hi(xa[e]), b0 = bf16lo(ya[e]), b1 = bf16hi(ya[e]);
        xa[e] = pack_bf16x2(a0 * t0.x - b0 * t0.y, a1 * t1.x - b1 * t1.y);
        ya[e] = pack_bf16x2(b0 * t0.x + a0 * t0.y, b1 * t1.x + a1 * t1.y);
      }
    }
    *reinterpret_cast<uint4*>(dst + i0) = x;
    *reinterpret_cast<uint4*>(dst + 64 + i0) = y;
  }
}

}  // namespace

cudaError_t launch_rope_table_axes(const int32_t* pos, int ldpos, int M, int half, const RopeAxes& f, float2* cs,
                                   cudaStream_t s) {
  long long grid = ((long long)M * half + 255) / 256;
  if (grid > 152 * 8) grid = 152 * 8;
  cudaError_t e = launch_k(rope_table_axes_kernel, dim3((unsigned)grid), dim3(256), 0, s, pos, ldpos, M, half, f, cs);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_kv_append(const KvAppendArgs& a, cudaStream_t s) {
  cudaError_t e = launch_k(kv_append_kernel, dim3(a.M), dim3(128), 0, s, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace spec
