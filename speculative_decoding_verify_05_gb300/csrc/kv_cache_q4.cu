// The paged cache in 4 bits (q4.cuh): norms of queries and keys with their rotation, the append that quantises a
// chunk's keys and values, and the read of cached keys and values.
#include "common.cuh"
#include "internal.h"
#include "paged_rows.cuh"
#include "q4.cuh"

namespace spec {
namespace {

constexpr int D = 128;
constexpr unsigned ALL = 0xffffffffu;

// ----------------------------------------------------------------- norm and rotation of a head
// Eight lanes hold a head: dims i0 .. i0 + 7 and 64 + i0 .. (i0 = 8 (lane % 8)), which the rotation turns into one another.
struct Head {
  float a[8], b[8];
};
__device__ __forceinline__ void unpack8(const uint4& x, float* v) {
  v[0] = bf16lo(x.x); v[1] = bf16hi(x.x); v[2] = bf16lo(x.y); v[3] = bf16hi(x.y);
  v[4] = bf16lo(x.z); v[5] = bf16hi(x.z); v[6] = bf16lo(x.w); v[7] = bf16hi(x.w);
}
__device__ __forceinline__ uint4 pack8(const float* v) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ float squares8(const float* v) {
  float p[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) p[e] = __fmul_rn(v[e], v[e]);
  return __fadd_rn(__fadd_rn(__fadd_rn(p[0], p[1]), __fadd_rn(p[2], p[3])),
                   __fadd_rn(__fadd_rn(p[4], p[5]), __fadd_rn(p[6], p[7])));
}
// y = x / sqrt(mean(x^2) + eps) * w.  The squares are summed neighbours first (1, 2, 4, .. 64 apart), and every
// operation is rounded once, so that a row's bytes in the cache do not depend on the chunk it came in or on which kernel
// normed it.  By all lanes of a warp.
__device__ __forceinline__ void norm_head(Head& h, const uint16_t* w, int i0, float eps) {
  float s0 = squares8(h.a), s1 = squares8(h.b);
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    s0 = __fadd_rn(s0, __shfl_xor_sync(ALL, s0, o));
    s1 = __fadd_rn(s1, __shfl_xor_sync(ALL, s1, o));
  }
  const float r = __frcp_rn(__fsqrt_rn(__fadd_rn(__fmul_rn(__fadd_rn(s0, s1), 1.f / D), eps)));
  float wa[8], wb[8];
  unpack8(__ldg(reinterpret_cast<const uint4*>(w + i0)), wa);
  unpack8(__ldg(reinterpret_cast<const uint4*>(w + 64 + i0)), wb);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    h.a[e] = __fmul_rn(__fmul_rn(h.a[e], r), wa[e]);
    h.b[e] = __fmul_rn(__fmul_rn(h.b[e], r), wb[e]);
  }
}
// (a, b) -> (a c - b s, b c + a s); t: (cos, sin) of dims i0 ..
__device__ __forceinline__ void turn_head(Head& h, const float4* t) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float c = (e & 1) ? t[e >> 1].z : t[e >> 1].x, s = (e & 1) ? t[e >> 1].w : t[e >> 1].y;
    const float a = h.a[e], b = h.b[e];
    h.a[e] = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
    h.b[e] = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  }
}
__device__ __forceinline__ void turns_of(const float2* cs, int r, int i0, float4* t) {
#pragma unroll
  for (int k = 0; k < 4; ++k) t[k] = __ldg(reinterpret_cast<const float4*>(cs + (size_t)r * 64 + i0) + k);
}

// One CTA per row; eight lanes per head, heads 4 WARPS apart.
template <int WARPS, int UNITS>
__global__ void __launch_bounds__(32 * WARPS) qk_norm_rope_kernel(const NormRopeArgs a) {
  constexpr int STEP = 4 * WARPS;
  pdl_wait();
  pdl_trigger();
  const int r = blockIdx.x, lane = threadIdx.x & 31, i0 = (lane & 7) * 8, heads = a.Hq + a.Hkv;
  float4 t[4];
  if (a.cs) turns_of(a.cs, r, i0, t);
  for (int h0 = (threadIdx.x >> 5) * 4; h0 < heads; h0 += STEP * UNITS) {
    uint4 x[UNITS], y[UNITS];
#pragma unroll
    for (int k = 0; k < UNITS; ++k) {
      const int hd = h0 + STEP * k + (lane >> 3);
      x[k] = y[k] = make_uint4(0, 0, 0, 0);
      if (hd >= heads) continue;
      const uint16_t* src = hd < a.Hq ? a.Q + (size_t)r * a.ldq + (size_t)hd * D
                                      : a.K + (size_t)r * a.ldk + (size_t)(hd - a.Hq) * D;
      x[k] = ld_past_l1(src + i0);
      y[k] = ld_past_l1(src + 64 + i0);
    }
#pragma unroll
    for (int k = 0; k < UNITS; ++k) {
      const int hd = h0 + STEP * k + (lane >> 3);
      if (h0 + STEP * k >= heads) continue;              // (the whole warp)
      Head h;
      unpack8(x[k], h.a);
      unpack8(y[k], h.b);
      norm_head(h, hd < a.Hq || a.Hkv == 0 ? a.wq : a.wk, i0, a.eps);    // (lanes past the last head: any weights)
      if (a.cs) turn_head(h, t);
      if (hd >= heads) continue;
      uint16_t* dst = hd < a.Hq ? a.Qout + (size_t)r * a.ldqo + (size_t)hd * D
                                : a.Kout + (size_t)r * a.ldko + (size_t)(hd - a.Hq) * D;
      st_past_l1(dst + i0, pack8(h.a));
      st_past_l1(dst + 64 + i0, pack8(h.b));
    }
  }
}

// ----------------------------------------------------------------- blocks of keys
// The keys of the sequences in aligned blocks of 2^LB (a word of values holds 8 keys): block v belongs to the last sequence
// whose first block, (cu_rows[b] >> LB) + 2 b, is at or before it.  A sequence's n rows lie in at most
// floor(n / 2^LB) + 2 blocks, which is what the sequences' first blocks are apart at least, so no walk over the
// batch is needed and (M >> LB) + 2 B blocks hold everyone.
struct Block {
  int b, page;                             // b -1: nothing
  int key0;                                // first key of the block
  int lo, hi;                              // its keys lo .. hi - 1 are rows of the sequence
  int row0;                                // packed row of key key0 + 0 (may be before the sequence's first)
};
template <int LB, class Args>
__device__ __forceinline__ Block block_of(int v, const Args& a, int lane, unsigned site) {
  Block k{-1, 0, 0, 0, 0, 0};
  const Place at = place_of(v, a, lane, [](int c0, int b) { return (c0 >> LB) + 2 * b; });
  if (at.b < 0 || at.c1 <= at.c0 || out_of_bounds(at.c0, at.c1, at.ctx, a)) return k;
  const long long key0 = ((long long)(at.ctx >> LB) + (v - ((at.c0 >> LB) + 2 * at.b))) << LB;
  const int end = at.ctx + (at.c1 - at.c0);
  if (key0 >= end) return k;
  k.key0 = (int)key0;
  k.lo = max(at.ctx - k.key0, 0);
  k.hi = min(end - k.key0, 1 << LB);
  k.row0 = at.c0 + (k.key0 - at.ctx);
  k.page = a.block_table[(size_t)at.b * a.max_pages + k.key0 / Q4_PAGE];
  if (k.page < 0 || k.page >= a.num_pages) {
    if (lane == 0) set_status(a.status, site);
    return k;
  }
  k.b = at.b;
  return k;
}
template <class Args>
__device__ __forceinline__ void check_sequence(const Args& a, long long b, unsigned site) {
  if (b < a.B && out_of_bounds(a.cu_rows[b], a.cu_rows[b + 1], a.ctx_len[b], a)) set_status(a.status, site);
}

// ----------------------------------------------------------------- append
// Values of a block of 8 keys of one kv head, by a warp: a lane has dims 4 lane .. 4 lane + 3 of all 8 keys, which are 4
// words of the page.  Entries of other keys in a word stay as they are (a page that receives rows belongs to
// one sequence, and a sequence's words each to one warp).
__device__ __forceinline__ void append_values(const KvAppendQ4Args& a, int v, int g, int lane) {
  const Block k = block_of<3>(v, a, lane, 0x8F2u);
  if (k.b < 0) return;
  uint8_t* page = a.Vpool + ((size_t)g * a.num_pages + k.page) * Q4_BYTES;
  const int slot = k.key0 % Q4_PAGE;
  uint32_t* words = reinterpret_cast<uint32_t*>(page + (slot >> 5) * Q4_PLANE + lane * 64) + ((slot >> 3) & 3);
  uint2 x[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    x[j] = make_uint2(0, 0);
    if (j >= k.lo && j < k.hi)
      x[j] = __ldg(reinterpret_cast<const uint2*>(a.Vnew + (size_t)(k.row0 + j) * a.ldkv + (size_t)g * D + lane * 4));
  }
  uint32_t w[4] = {0, 0, 0, 0}, mask = 0;
  const bool part = k.hi - k.lo < 8;
  if (part) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < k.lo || j >= k.hi) mask |= 15u << q4_shift(j);
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = words[4 * e] & mask;
  }
  unsigned mine = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (j < k.lo || j >= k.hi) continue;
    const float f[4] = {bf16lo(x[j].x), bf16hi(x[j].x), bf16lo(x[j].y), bf16hi(x[j].y)};
    float top = fmaxf(fmaxf(fabsf(f[0]), fabsf(f[1])), fmaxf(fabsf(f[2]), fabsf(f[3])));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) top = fmaxf(top, __shfl_xor_sync(ALL, top, o));
    unsigned code;
    const float s = q4_scale(top, code);
    if ((lane & 7) == j) mine = code;
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] |= q4_entry(f[e], s) << q4_shift(j);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) words[4 * e] = w[e];
  const int j = lane & 7;
  if (j >= k.lo && j < k.hi) page[Q4_SCALES + (lane >> 3) * 128 + slot + j] = (uint8_t)mine;
}

// Keys, of eight lanes with a head: a lane's two runs of 8 dims are a word each, four lanes have a scale together.
__device__ __forceinline__ void append_key(const KvAppendQ4Args& a, const Head& h, int g, int page, int slot, int lane,
                                           bool used) {
  float ta = 0.f, tb = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    ta = fmaxf(ta, fabsf(h.a[e]));
    tb = fmaxf(tb, fabsf(h.b[e]));
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    ta = fmaxf(ta, __shfl_xor_sync(ALL, ta, o));
    tb = fmaxf(tb, __shfl_xor_sync(ALL, tb, o));
  }
  unsigned ca, cb;
  const float sa = q4_scale(ta, ca), sb = q4_scale(tb, cb);
  uint32_t wa = 0, wb = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    wa |= q4_entry(h.a[e], sa) << q4_shift(e);
    wb |= q4_entry(h.b[e], sb) << q4_shift(e);
  }
  // scales of dims 0, 32, 64, 96 ..: lanes 0 and 4 of the eight
  const unsigned mine = ca | (cb << 16), codes = mine | (__shfl_xor_sync(ALL, mine, 4) << 8);
  if (!used) return;
  uint8_t* p = a.Kpool + ((size_t)g * a.num_pages + page) * Q4_BYTES;
  const int l = lane & 7;
  uint32_t* word = reinterpret_cast<uint32_t*>(p + (l >> 2) * Q4_PLANE + slot * 16) + (l & 3);
  word[0] = wa;
  word[2 * Q4_PLANE / 4] = wb;
  if (l == 0) reinterpret_cast<uint32_t*>(p + Q4_SCALES)[slot] = codes;
}

// CTAs: one per row for its queries and keys, then four blocks of values each, then a thread per sequence that checks its
// bounds (no row has to be in a sequence that breaks them).
template <int WARPS, int UNITS>
__global__ void __launch_bounds__(32 * WARPS) kv_append_q4_kernel(const KvAppendQ4Args a) {
  constexpr int STEP = 4 * WARPS;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, i0 = (lane & 7) * 8;
  const int r = blockIdx.x;
  if (r >= a.M) {
    const unsigned u = (unsigned)(r - a.M) * WARPS + warp, units = (unsigned)a.blocks * a.Hkv;
    const unsigned ctas = (units + WARPS - 1) / WARPS;
    if ((unsigned)(r - a.M) < ctas) {
      if (u < units) append_values(a, u / a.Hkv, u % a.Hkv, lane);
    } else {
      check_sequence(a, (long long)(r - a.M - ctas) * (32 * WARPS) + threadIdx.x, 0x8F1u);
    }
    return;
  }
  const int heads = a.Hq + a.Hkv;
  float4 t[4];
  if (a.cs) turns_of(a.cs, r, i0, t);
  int b = -2, page = 0, p = 0;
  for (int h0 = warp * 4; h0 < heads || b == -2; h0 += STEP * UNITS) {
    uint4 x[UNITS], y[UNITS];
#pragma unroll
    for (int k = 0; k < UNITS; ++k) {
      const int hd = h0 + STEP * k + (lane >> 3);
      x[k] = y[k] = make_uint4(0, 0, 0, 0);
      if (hd >= heads) continue;
      const uint16_t* src = hd < a.Hq ? a.Q + (size_t)r * a.ldq + (size_t)hd * D
                                      : a.Knew + (size_t)r * a.ldkv + (size_t)(hd - a.Hq) * D;
      x[k] = ld_past_l1(src + i0);
      y[k] = ld_past_l1(src + 64 + i0);
    }
    if (b == -2) {                                      // the row's sequence, position and page
      const Place at = place_of(r, a, lane);
      b = at.b;
      if (b < 0 || r >= at.c1) return;                  // padding
      if (out_of_bounds(at.c0, at.c1, at.ctx, a)) return;
      p = at.ctx + (r - at.c0);
      page = a.block_table[(size_t)b * a.max_pages + p / Q4_PAGE];
      if (page < 0 || page >= a.num_pages) {
        if (threadIdx.x == 0) set_status(a.status, 0x8F2u);
        page = -1;
      }
    }
#pragma unroll
    for (int k = 0; k < UNITS; ++k) {
      const int hd = h0 + STEP * k + (lane >> 3);
      if (h0 + STEP * k >= heads) continue;             // (the whole warp)
      Head h;
      unpack8(x[k], h.a);
      unpack8(y[k], h.b);
      if (a.wk) norm_head(h, hd < a.Hq ? a.wq : a.wk, i0, a.eps);      // (wq is there if Hq > 0)
      if (a.cs) turn_head(h, t);
      const bool is_q = hd < a.Hq;
      if (is_q) {
        uint16_t* dst = a.Qrot + (size_t)r * a.ldqr + (size_t)hd * D;
        st_past_l1(dst + i0, pack8(h.a));
        st_past_l1(dst + 64 + i0, pack8(h.b));
      }
      if (__any_sync(ALL, !is_q)) append_key(a, h, hd - a.Hq, page, p % Q4_PAGE, lane, !is_q && hd < heads && page >= 0);
    }
  }
}

// ----------------------------------------------------------------- read
// A warp per 32 keys of one kv head.  Keys: eight lanes per key, a lane's two words of 8 dims.  Values: a lane has dims
// 4 lane .. 4 lane + 3 of all 32 keys (16 bytes of the page each), so that a key's 128 dims leave as one line.
__global__ void __launch_bounds__(128) kv_read_q4_kernel(const KvReadQ4Args a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const unsigned units = (unsigned)a.blocks * a.Hkv, ctas = (units + 3) / 4;
  const unsigned u = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (blockIdx.x >= ctas) {
    check_sequence(a, (long long)(blockIdx.x - ctas) * 128 + threadIdx.x, 0x9F1u);
    return;
  }
  if (u >= units) return;
  const int g = u % a.Hkv;
  const Block k = block_of<5>(u / a.Hkv, a, lane, 0x9F2u);
  if (k.b < 0) return;
  const size_t at = ((size_t)g * a.num_pages + k.page) * Q4_BYTES;
  const int slot0 = k.key0 % Q4_PAGE;
  // values first: their loads are the longer wait
  const uint8_t* vp = a.Vpool + at;
  uint4 vw[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    vw[e] = *reinterpret_cast<const uint4*>(vp + (slot0 >> 5) * Q4_PLANE + (lane * 4 + e) * 16);
  uint4 vc[2];
#pragma unroll
  for (int e = 0; e < 2; ++e)
    vc[e] = *reinterpret_cast<const uint4*>(vp + Q4_SCALES + (lane >> 3) * 128 + slot0 + 16 * e);
  const uint8_t* kp = a.Kpool + at;
  const int l = lane & 7;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int j = 4 * i + (lane >> 3), slot = slot0 + j;
    if (j < k.lo || j >= k.hi) continue;
    const uint32_t* word = reinterpret_cast<const uint32_t*>(kp + (l >> 2) * Q4_PLANE + slot * 16) + (l & 3);
    const uint32_t wa = word[0], wb = word[2 * Q4_PLANE / 4];
    const uint32_t codes = reinterpret_cast<const uint32_t*>(kp + Q4_SCALES)[slot] >> (8 * (l >> 2));
    const uint32_t sa = q4_scale2((codes & 255u) * 0x10001u), sb = q4_scale2(((codes >> 16) & 255u) * 0x10001u);
    const uint32_t oa = q4_offset2(sa), ob = q4_offset2(sb);
    uint16_t* dst = a.Kout + (size_t)(k.row0 + j) * a.ldkv + (size_t)g * D + l * 8;
    st_past_l1(dst, make_uint4(q4_pair<0>(wa, sa, oa), q4_pair<1>(wa, sa, oa), q4_pair<2>(wa, sa, oa),
                               q4_pair<3>(wa, sa, oa)));
    st_past_l1(dst + 64, make_uint4(q4_pair<0>(wb, sb, ob), q4_pair<1>(wb, sb, ob), q4_pair<2>(wb, sb, ob),
                                    q4_pair<3>(wb, sb, ob)));
  }
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    if (j < k.lo || j >= k.hi) continue;
    const uint32_t cw = reinterpret_cast<const uint32_t*>(vc)[j >> 2];
    const uint32_t s = q4_scale2(((cw >> (8 * (j & 3))) & 255u) * 0x10001u), o = q4_offset2(s);
    uint32_t n[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) n[e] = (reinterpret_cast<const uint32_t*>(&vw[e])[j >> 3] >> q4_shift(j & 7)) & 15u;
    const uint2 out = make_uint2(q4_fma2(n[0] | (n[1] << 16) | 0x43004300u, s, o),
                                 q4_fma2(n[2] | (n[3] << 16) | 0x43004300u, s, o));
    *reinterpret_cast<uint2*>(a.Vout + (size_t)(k.row0 + j) * a.ldkv + (size_t)g * D + lane * 4) = out;
  }
}

}  // namespace

cudaError_t launch_qk_norm_rope(const NormRopeArgs& a, int sms, cudaStream_t s) {
  const bool many = a.M > 10 * sms;
  auto* k = many ? qk_norm_rope_kernel<2, 2> : qk_norm_rope_kernel<4, 3>;
  cudaError_t e = launch_k(k, dim3((unsigned)a.M), dim3(many ? 64 : 128), 0, s, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_kv_append_q4(const KvAppendQ4Args& args, int sms, cudaStream_t s) {
  KvAppendQ4Args a = args;
  const bool many = a.M > 10 * sms;
  const unsigned warps = many ? 2 : 4;
  a.blocks = (a.M >> 3) + 2 * a.B;
  const unsigned values = ((unsigned)a.blocks * a.Hkv + warps - 1) / warps, checks = ((unsigned)a.B + 32 * warps - 1) / (32 * warps);
  auto* k = many ? kv_append_q4_kernel<2, 2> : kv_append_q4_kernel<4, 3>;
  cudaError_t e = launch_k(k, dim3((unsigned)a.M + values + checks), dim3(32 * warps), 0, s, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_kv_read_q4(const KvReadQ4Args& args, cudaStream_t s) {
  KvReadQ4Args a = args;
  a.blocks = (a.M >> 5) + 2 * a.B;
  const unsigned units = ((unsigned)a.blocks * a.Hkv + 3) / 4, checks = ((unsigned)a.B + 127) / 128;
  cudaError_t e = launch_k(kv_read_q4_kernel, dim3(units + checks), dim3(128), 0, s, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace spec
