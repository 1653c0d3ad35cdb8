// Attention of a chunk of new tokens over the paged cache: row j of sequence b attends keys
// 0 .. ctx_b + j of its pages.
//
// One warp per (row, query head), four dims per lane, one pass over the keys with the running
// maximum and sum.
#include "common.cuh"
#include "internal.h"

namespace spec {
namespace {

constexpr int D = 128;
constexpr int PAGE = 128;

__global__ void __launch_bounds__(128) chunk_attention_kernel(const ChunkAttnArgs a) {
  pdl_wait();
  pdl_trigger();
  const int r = blockIdx.x, h = blockIdx.y * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  int lo = 0, hi = a.B - 1;
  while (lo < hi) {                     // the last sequence with cu_rows[b] <= r
    const int mid = (lo + hi + 1) >> 1;
    if (a.cu_rows[mid] <= r) lo = mid; else hi = mid - 1;
  }
  const int c0 = a.cu_rows[lo], c1 = a.cu_rows[lo + 1], ctx = a.ctx_len[lo];
  if (r < c0 || r >= c1 || h >= a.Hkv * a.G) return;
  if (c0 < 0 || c1 > a.M || ctx < 0 || (long long)ctx + (c1 - c0) > (long long)a.max_pages * PAGE) {
    if (threadIdx.x == 0) set_status(a.status, 0x7F1u);
    return;
  }
  const int keys = ctx + (r - c0) + 1, g = h / a.G;
  const uint2 qv = *reinterpret_cast<const uint2*>(a.Q + (size_t)r * a.ldq + (size_t)h * D + lane * 4);
  const float q0 = bf16lo(qv.x), q1 = bf16hi(qv.x), q2 = bf16lo(qv.y), q3 = bf16hi(qv.y);
  float m = -INFINITY, l = 0.f, o0 = 0.f, o1 = 0.f, o2 = 0.f, o3 = 0.f;
  for (int t = 0; t * PAGE < keys; ++t) {
    int page = a.block_table[(size_t)lo * a.max_pages + t];
    if (page < 0 || page >= a.num_pages) {
      if (lane == 0) set_status(a.status, 0x7F2u);
      page = 0;
    }
    const size_t base = ((size_t)g * a.num_pages + page) * PAGE * D + lane * 4;
    const int n = min(PAGE, keys - t * PAGE);
    for (int k = 0; k < n; ++k) {
      const uint2 kv = *reinterpret_cast<const uint2*>(a.Kpool + base + (size_t)k * D);
      const uint2 vv = *reinterpret_cast<const uint2*>(a.Vpool + base + (size_t)k * D);
      float x = q0 * bf16lo(kv.x) + q1 * bf16hi(kv.x) + q2 * bf16lo(kv.y) + q3 * bf16hi(kv.y);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      x *= a.scale_log2;
      const float mn = fmaxf(m, x), f = exp2f(m - mn), e = exp2f(x - mn);
      m = mn;
      l = l * f + e;
      o0 = o0 * f + e * bf16lo(vv.x);
      o1 = o1 * f + e * bf16hi(vv.x);
      o2 = o2 * f + e * bf16lo(vv.y);
      o3 = o3 * f + e * bf16hi(vv.y);
    }
  }
  const float inv = 1.f / l;
  *reinterpret_cast<uint2*>(a.O + (size_t)r * a.ldo + (size_t)h * D + lane * 4) =
      make_uint2(pack_bf16x2(o0 * inv, o1 * inv), pack_bf16x2(o2 * inv, o3 * inv));
}

}  // namespace

cudaError_t launch_chunk_attention(const ChunkAttnArgs& a, cudaStream_t s) {
  cudaError_t e = launch_k(chunk_attention_kernel, dim3(a.M, (a.Hkv * a.G + 3) / 4), dim3(128), 0, s, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace spec
