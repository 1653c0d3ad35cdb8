// Prompt side of the paged cache, the two kernels before the attention of a chunk: the rotation table
// of positions with several axes, and the append of a chunk's keys and values to their pages with the
// rotation applied on the way.
#include "common.cuh"
#include "internal.h"
#include "paged_rows.cuh"

namespace spec {
namespace {

constexpr int D = 128;
constexpr int PAGE = 128;

// (cos, sin) of u / 2^64 turns.  The position times the frequency is formed modulo one turn in 64-bit integers
// (wrap-around is the reduction, exact for any 32-bit position), the nearest quarter turn is split off,
// and what is left, at most an eighth of a turn, is off by less than 2^-32 turns (the low word is dropped) before its
// one rounding to fp32.  There
// the Taylor series of sin(pi x) and cos(pi x) on |x| <= 1/4 (terms to (pi x)^9 and (pi x)^10: the next are below
// 2e-9) take 11 multiply-adds; sincospif, which has the whole line to care for, took 1.7 us
// more for the 16000-row table.  No fp64 instruction: the chip has few of them.
__device__ __forceinline__ float2 cos_sin_turns(unsigned long long u) {
  const unsigned hi = (unsigned)(u >> 32);
  const unsigned quarter = (hi + (1u << 29)) >> 30;                 // 0..4, 4 = 0
  const float x = (float)(int)(hi - (quarter << 30)) * 0x1p-31f;    // 2 pi rem / 2^32 = pi (rem / 2^31)
  const float z = x * x;
  // pi^k / k!; pi in two parts
  float s = 0.08214588661112822879880237f;
  s = fmaf(s, z, -0.5992645293207919f);
  s = fmaf(s, z, 2.550164039877345f);
  s = fmaf(s, z, -5.167712780049969f);
  s = fmaf(s, z, -8.742278012618954e-8f);
  s = fmaf(x, 3.1415927410125732421875f, x * s);
  float c = -0.02580689139001405f;
  c = fmaf(c, z, 0.23533063035889312f);
  c = fmaf(c, z, -1.3352627688545893f);
  c = fmaf(c, z, 4.058712126416768f);
  c = fmaf(c, z, -4.934802200544679f);
  c = fmaf(c, z, 1.f);
  // a quarter turn maps (c, s) to (-s, c)
  const float a = (quarter & 1u) ? s : c, b = (quarter & 1u) ? c : s;
  return make_float2(((quarter + 1u) & 2u) ? -a : a, (quarter & 2u) ? -b : b);
}

// A thread keeps one frequency and walks `rows` rows with it.  Its turn and axis are parameters, read by ordinary
// loads (the pointers' origin hidden from the compiler): from the parameter bank 32 lanes with 32 addresses are served
// one after the other, for every CTA anew (16000 rows of 64 frequencies 4.2 us instead of 3.3; per entry, with
// integer divisions, 16.4).
template <typename T>
__device__ __forceinline__ const T* as_memory(const T* p) {
  asm volatile("" : "+l"(p));
  return p;
}
__global__ void __launch_bounds__(256)
rope_table_axes_kernel(const int32_t* __restrict__ pos, int ldpos, int M, int half, int rows,
                       const __grid_constant__ RopeAxes f, float2* __restrict__ cs) {
  pdl_wait();
  pdl_trigger();
  const int i = threadIdx.x;
  if (i >= half) return;
  const unsigned long long turn = as_memory(f.turn)[i];
  const int32_t* p = pos + (size_t)as_memory(f.axis)[i] * ldpos;
  const unsigned r0 = (blockIdx.x * blockDim.y + threadIdx.y) * rows, r1 = min(r0 + rows, (unsigned)M);
#pragma unroll 4
  for (unsigned r = r0; r < r1; ++r) cs[(size_t)r * half + i] = cos_sin_turns((unsigned long long)(long long)p[r] * turn);
}

// One CTA per row, and behind them a thread per sequence that checks its bounds (no row has to be in a sequence that
// breaks them).  A thread of a row moves pairs of 16-byte chunks (dims i0 .. and 64 + i0 ..) of heads 4 WARPS apart, so
// its eight angles stay in registers; up to UNITS pairs are loaded before the row's place in the cache is known,
// which takes two dependent loads.  Bound by HBM: 8192 rows of 32 + 2 x 8 heads, 206 MB, take 32.9 us (6.3 TB/s),
// 24 sequences of 1 to 999 rows, 81 MB, 13.9 us (5.8).
// Two shapes.  Few rows: a row's whole traffic in flight at once, 4 warps and up to 4 pairs (8 rows 2.5 us, 1000 rows
// 4.4; the other shape 3.3 and 5.3).  Many rows: CTAs that are small enough for 16 and more to share an SM, so that
// some move data while others look their place up (8192 rows 32.9 us, the 24 sequences 14.2; the other shape
// 33.8 and 17.3).  The two meet at 10 rows per SM (1500 rows: 8.4 us both).
// Stores go past L1 (3600 rows of keys and values 5.4 -> 4.7 us, none slower); loads only where many rows are turned
// (the 24 sequences 14.2 -> 13.9 us; the copy of 3600 rows would take 5.3).
template <int WARPS, int UNITS, bool TURN>
__global__ void __launch_bounds__(32 * WARPS) kv_append_kernel(const KvAppendArgs a) {
  constexpr int STEP = 4 * WARPS;                       // heads between a thread's pairs
  constexpr bool LOAD_PAST_L1 = WARPS == 2 && TURN;
  pdl_wait();
  pdl_trigger();
  const int r = blockIdx.x, tid = threadIdx.x, i0 = (tid & 7) * 8;
  if (r >= a.M) {
    const long long b = (long long)(r - a.M) * (32 * WARPS) + tid;
    if (b < a.B && out_of_bounds(a.cu_rows[b], a.cu_rows[b + 1], a.ctx_len[b], a)) set_status(a.status, 0x6F1u);
    return;
  }
  const int heads = a.Hq + 2 * a.Hkv;
  float4 t[4];                                          // (cos, sin) of dims i0 ..
  if constexpr (TURN)
#pragma unroll
    for (int k = 0; k < 4; ++k) t[k] = *(reinterpret_cast<const float4*>(a.cs + (size_t)r * 64 + i0) + k);
  int b = -2, page = 0, p = 0;
  for (int h0 = tid >> 3; h0 < heads || b == -2; h0 += STEP * UNITS) {
    uint4 x[UNITS], y[UNITS];
#pragma unroll
    for (int k = 0; k < UNITS; ++k) {
      const int hd = h0 + STEP * k;
      if (hd >= heads) continue;
      const uint16_t* src;
      if (hd < a.Hq) src = a.Q + (size_t)r * a.ldq + (size_t)hd * D;
      else if (hd < a.Hq + a.Hkv) src = a.Knew + (size_t)r * a.ldkv + (size_t)(hd - a.Hq) * D;
      else src = a.Vnew + (size_t)r * a.ldkv + (size_t)(hd - a.Hq - a.Hkv) * D;
      x[k] = LOAD_PAST_L1 ? ld_past_l1(src + i0) : *reinterpret_cast<const uint4*>(src + i0);
      y[k] = LOAD_PAST_L1 ? ld_past_l1(src + 64 + i0) : *reinterpret_cast<const uint4*>(src + 64 + i0);
    }
    if (b == -2) {                                      // the row's sequence, position and page
      const Place at = place_of(r, a, tid & 31);
      b = at.b;
      if (b < 0 || r >= at.c1) return;                  // padding
      if (out_of_bounds(at.c0, at.c1, at.ctx, a)) return;
      p = at.ctx + (r - at.c0);
      page = a.block_table[(size_t)b * a.max_pages + p / PAGE];
      if (page < 0 || page >= a.num_pages) {
        if (tid == 0) set_status(a.status, 0x6F2u);
        page = -1;
      }
    }
#pragma unroll
    for (int k = 0; k < UNITS; ++k) {
      const int hd = h0 + STEP * k;
      if (hd >= heads) continue;
      const bool is_v = hd >= a.Hq + a.Hkv;
      uint16_t* dst;
      if (hd < a.Hq) {
        dst = a.Qrot + (size_t)r * a.ldqr + (size_t)hd * D;
      } else {
        if (page < 0) continue;
        const int g = hd - a.Hq - (is_v ? a.Hkv : 0);
        dst = (is_v ? a.Vpool : a.Kpool) + (((size_t)g * a.num_pages + page) * PAGE + p % PAGE) * D;
      }
      if (TURN && !is_v) {
        uint32_t* xa = reinterpret_cast<uint32_t*>(&x[k]);
        uint32_t* ya = reinterpret_cast<uint32_t*>(&y[k]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float a0 = bf16lo(xa[e]), a1 = bf16hi(xa[e]), b0 = bf16lo(ya[e]), b1 = bf16hi(ya[e]);
          xa[e] = pack_bf16x2(a0 * t[e].x - b0 * t[e].y, a1 * t[e].z - b1 * t[e].w);
          ya[e] = pack_bf16x2(b0 * t[e].x + a0 * t[e].y, b1 * t[e].z + a1 * t[e].w);
        }
      }
      st_past_l1(dst + i0, x[k]);
      st_past_l1(dst + 64 + i0, y[k]);
    }
  }
}

}  // namespace

cudaError_t launch_rope_table_axes(const int32_t* pos, int ldpos, int M, int half, const RopeAxes& f, float2* cs, int sms,
                                   cudaStream_t s) {
  // rows per thread: one while that fills the chip, more (up to 8) when there are many
  const int bx = (half + 31) / 32 * 32, by = bx < 256 ? 256 / bx : 1;
  const int fill = M / (by * sms * 2), rows = fill < 1 ? 1 : (fill > 8 ? 8 : fill);
  cudaError_t e = launch_k(rope_table_axes_kernel, dim3(((unsigned)M + by * rows - 1) / (by * rows)), dim3(bx, by), 0, s,
                           pos, ldpos, M, half, rows, f, cs);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_kv_append(const KvAppendArgs& a, int sms, cudaStream_t s) {
  const bool many = a.M > 10 * sms;
  const dim3 block(many ? 64 : 128);
  auto* turn = many ? kv_append_kernel<2, 2, true> : kv_append_kernel<4, 4, true>;
  auto* copy = many ? kv_append_kernel<2, 2, false> : kv_append_kernel<4, 4, false>;
  const unsigned checks = ((unsigned)a.B + block.x - 1) / block.x;
  cudaError_t e = launch_k(a.cs ? turn : copy, dim3((unsigned)a.M + checks), block, 0, s, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace spec
