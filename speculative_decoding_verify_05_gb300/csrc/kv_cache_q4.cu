// The paged cache in 4 bits (q4.cuh): norms of queries and keys with their rotation, the append that quantises a
// chunk's keys and values, and the read of cached keys and values.
//
// Bound.  Of a few rows, a launch and the chain of loads behind it (norm of 9 rows 3.5 us, append of 8 4.1, read of 77
// keys 4.2: lengths, page id, page, output).  Of many, with 32 / 8 heads, in bytes of inputs and outputs:
//   norm, 8192 rows    29.7 us = 5.8 TB/s, 87 % of the copy; loads wait for HBM (issue 50 %)
//   append, 8192 rows  38.8 us = 4.7 TB/s, 70 %; issue 59 %: some 15 instructions a value for norm, rotation, maximum,
//                      quotient and packing, and chains of shuffles.  Keys and values alone take 14.7 us, which
//                      wait for instructions, the queries' share of the norm above 24, which waits for HBM: the grid
//                      has the one before the other, and the times add up
//   read, 32 contexts  62.4 us = 6.1 TB/s, 92 %
#include "attention_util.cuh"
#include "internal.h"
#include "paged_rows.cuh"
#include "q4.cuh"

namespace spec {
namespace {

constexpr int D = 128;
constexpr unsigned ALL = 0xffffffffu;

// ----------------------------------------------------------------- norm and rotation of a head
// Eight lanes hold a head: dims i0 .. i0 + 7 and 64 + i0 .. (i0 = 8 (lane % 8)), which the rotation turns into one another,
// as pairs, on which the packed fp32 instructions work (each half rounded as by itself, so every operation is rounded
// once; 8192 rows of 32 + 8 heads 37.1 us without).
struct Head {
  float2 v[8];
};
__device__ __forceinline__ Head head_of(const uint4& x, const uint4& y) {
  Head h;
  const uint32_t a[4] = {x.x, x.y, x.z, x.w}, b[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    h.v[2 * e] = make_float2(bf16lo(a[e]), bf16lo(b[e]));
    h.v[2 * e + 1] = make_float2(bf16hi(a[e]), bf16hi(b[e]));
  }
  return h;
}
__device__ __forceinline__ void store_head(uint16_t* dst, const Head& h) {
  uint32_t a[4], b[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    a[e] = cvt_bf16x2(h.v[2 * e].x, h.v[2 * e + 1].x);
    b[e] = cvt_bf16x2(h.v[2 * e].y, h.v[2 * e + 1].y);
  }
  st_past_l1(dst, make_uint4(a[0], a[1], a[2], a[3]));
  st_past_l1(dst + 64, make_uint4(b[0], b[1], b[2], b[3]));
}
// y = x / sqrt(mean(x^2) + eps) * w.  The squares are summed neighbours first (1, 2, 4, .. 64 apart), so that a row's bytes
// in the cache do not depend on the chunk it came in or on which kernel normed it.  By all lanes of a warp; w: the
// weights, as head_of has them.
__device__ __forceinline__ void norm_head(Head& h, const Head& w, float eps) {
  float2 p[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) p[e] = q4_mul2(h.v[e], h.v[e]);
  float2 s = add2(add2(add2(p[0], p[1]), add2(p[2], p[3])), add2(add2(p[4], p[5]), add2(p[6], p[7])));
#pragma unroll
  for (int o = 1; o < 8; o <<= 1)
    s = add2(s, make_float2(__shfl_xor_sync(ALL, s.x, o), __shfl_xor_sync(ALL, s.y, o)));
  const float r = __frcp_rn(__fsqrt_rn(__fadd_rn(__fmul_rn(__fadd_rn(s.x, s.y), 1.f / D), eps)));
#pragma unroll
  for (int e = 0; e < 8; ++e) h.v[e] = q4_mul2(q4_mul2(h.v[e], make_float2(r, r)), w.v[e]);
}
// (a, b) -> (a c - b s, b c + a s), each product rounded before the sum.  The sums are __fadd_rn, which is never merged with a
// product; a packed add of packed products was compiled to a multiply-add, in which a c stays unrounded (16 of a million
// bf16 results were off by a step).
struct Turns {
  float c[8], s[8];
};
__device__ __forceinline__ void turn_head(Head& h, const Turns& t) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float2 x = q4_mul2(h.v[e], make_float2(t.c[e], t.c[e]));
    const float2 y = q4_mul2(make_float2(h.v[e].y, h.v[e].x), make_float2(-t.s[e], t.s[e]));
    h.v[e] = make_float2(__fadd_rn(x.x, y.x), __fadd_rn(x.y, y.y));
  }
}
__device__ __forceinline__ Turns turns_of(const float2* cs, int r, int i0) {
  Turns t;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float4 u = __ldg(reinterpret_cast<const float4*>(cs + (size_t)r * 64 + i0) + k);
    t.c[2 * k] = u.x;
    t.s[2 * k] = u.y;
    t.c[2 * k + 1] = u.z;
    t.s[2 * k + 1] = u.w;
  }
  return t;
}

// The heads `heads` of one row (row r's at src), four to a warp, UNITS rounds of the CTA's warps under way at once: normed (w
// not null), rotated (turn), and handed to put(head number, head) by whole warps (heads >= `heads` are void).
template <int WARPS, int UNITS, class Before, class Put>
__device__ __forceinline__ void each_head(const uint16_t* src, int heads, const uint16_t* w, float eps, bool turn,
                                          const Turns& t, Before&& before, Put&& put) {
  constexpr int STEP = 4 * WARPS;
  const int lane = threadIdx.x & 31, i0 = (lane & 7) * 8;
  Head wh;
  if (w) wh = head_of(__ldg(reinterpret_cast<const uint4*>(w + i0)), __ldg(reinterpret_cast<const uint4*>(w + 64 + i0)));
  for (int h0 = (threadIdx.x >> 5) * 4; h0 < heads; h0 += STEP * UNITS) {
    uint4 x[UNITS], y[UNITS];
#pragma unroll
    for (int k = 0; k < UNITS; ++k) {
      const int hd = h0 + STEP * k + (lane >> 3);
      x[k] = y[k] = make_uint4(0, 0, 0, 0);
      if (hd >= heads) continue;
      x[k] = ld_past_l1(src + (size_t)hd * D + i0);
      y[k] = ld_past_l1(src + (size_t)hd * D + 64 + i0);
    }
    if (!before()) return;
#pragma unroll
    for (int k = 0; k < UNITS; ++k) {
      if (h0 + STEP * k >= heads) continue;              // (the whole warp)
      Head h = head_of(x[k], y[k]);
      if (w) norm_head(h, wh, eps);
      if (turn) turn_head(h, t);
      put(h0 + STEP * k + (lane >> 3), h);
    }
  }
}

// One CTA per row.  At least 14 CTAs of two warps an SM (72 registers a thread): 8192 rows 29.7 us, 3.4 more without the bound.
template <int WARPS, int UNITS>
__global__ void __launch_bounds__(32 * WARPS, WARPS == 2 ? 14 : 5) qk_norm_rope_kernel(const NormRopeArgs a) {
  pdl_wait();
  pdl_trigger();
  const int r = blockIdx.x, i0 = (threadIdx.x & 7) * 8;
  Turns t;
  if (a.cs) t = turns_of(a.cs, r, i0);
  auto nothing = []() { return true; };
  each_head<WARPS, UNITS>(a.Q + (size_t)r * a.ldq, a.Hq, a.wq, a.eps, a.cs != nullptr, t, nothing, [&](int hd, const Head& h) {
    if (hd < a.Hq) store_head(a.Qout + (size_t)r * a.ldqo + (size_t)hd * D + i0, h);
  });
  each_head<WARPS, 1>(a.K + (size_t)r * a.ldk, a.Hkv, a.wk, a.eps, a.cs != nullptr, t, nothing, [&](int hd, const Head& h) {
    if (hd < a.Hkv) store_head(a.Kout + (size_t)r * a.ldko + (size_t)hd * D + i0, h);
  });
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
__device__ __forceinline__ Block block_of(int v, const Args& a, int lane) {
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
  k.b = at.b;
  return k;
}
// (apart, so that loads that need no page are issued before its id is there: append of 8192 rows 0.9 us more otherwise)
template <class Args>
__device__ __forceinline__ bool page_exists(const Block& k, const Args& a, int lane, unsigned site) {
  const bool yes = k.page >= 0 && k.page < a.num_pages;
  if (!yes && lane == 0) set_status(a.status, site);
  return yes;
}
template <class Args>
__device__ __forceinline__ void check_sequence(const Args& a, long long b, unsigned site) {
  if (b < a.B && out_of_bounds(a.cu_rows[b], a.cu_rows[b + 1], a.ctx_len[b], a)) set_status(a.status, site);
}

// ----------------------------------------------------------------- append
// What eight keys of any values, infinities and NaN among them, add to a lane's four words; returns the code of key lane % 8.
// Out of line: seldom needed.
__device__ __noinline__ unsigned any_values(const uint2 (&x)[8], uint32_t (&add)[4]) {
  unsigned mine = 0;
  add[0] = add[1] = add[2] = add[3] = 0;
#pragma unroll 1
  for (int j = 0; j < 8; ++j) {
    const uint2 r = q4_any(make_float4(bf16lo(x[j].x), bf16hi(x[j].x), bf16lo(x[j].y), bf16hi(x[j].y)),
                           make_float4(0.f, 0.f, 0.f, 0.f), 8);
#pragma unroll
    for (int e = 0; e < 4; ++e) add[e] += (((r.x >> (4 * e)) & 15u) - 8u) << q4_shift(j);
    if ((threadIdx.x & 7) == j) mine = r.y;
  }
  return mine;
}

// Values of a block of 2^LB keys (8 or 32) of one kv head, by a warp: a lane has dims 4 lane .. 4 lane + 3 of all of them, which
// are one word or all four words of four rows of the page.  Entries of other keys in a word stay as they are (a
// page that receives rows belongs to one sequence, and a sequence's words each to one warp).
template <int LB>
__device__ __forceinline__ void append_values(const KvAppendQ4Args& a, int v, int g, int lane) {
  constexpr int WORDS = 1 << (LB - 3);
  const Block k = block_of<LB>(v, a, lane);
  if (k.b < 0) return;
  const uint16_t* src = a.Vnew + (size_t)g * D + lane * 4;
  uint32_t w[WORDS][4];
  auto load = [&](int i, uint2 (&x)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[j] = make_uint2(0, 0);
      const int key = 8 * i + j;
      if (key >= k.lo && key < k.hi) x[j] = __ldg(reinterpret_cast<const uint2*>(src + (size_t)(k.row0 + key) * a.ldkv));
    }
  };
  uint2 x[8];
  load(0, x);
  if (!page_exists(k, a, lane, 0x8F2u)) return;
  uint8_t* page = a.Vpool + ((size_t)g * a.num_pages + k.page) * Q4_BYTES;
  const int slot = k.key0 % Q4_PAGE;
  uint32_t* words = reinterpret_cast<uint32_t*>(page + (slot >> 5) * Q4_PLANE + lane * 64) + ((slot >> 3) & 3);
#pragma unroll
  for (int i = 0; i < WORDS; ++i) {
    uint2 next[8];
    if (i + 1 < WORDS) load(i + 1, next);
    const int lo = k.lo - 8 * i, hi = k.hi - 8 * i;
    uint32_t keep = 0;                     // entries of other keys
    if (lo > 0 || hi < 8) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < lo || j >= hi) keep |= 15u << q4_shift(j);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) w[i][e] = (keep ? words[4 * e + i] & keep : 0u) | (0x88888888u & ~keep);
    // (keys of other chunks and sequences are zeros here, which add nothing)
    unsigned top[8], mine;                 // (as bits: NaN lies above everything)
#pragma unroll
    for (int j = 0; j < 8; ++j)
      top[j] = max(max((x[j].x << 16) & 0x7fffffffu, x[j].x & 0x7fffffffu), max((x[j].y << 16) & 0x7fffffffu, x[j].y & 0x7fffffffu));
    // folded over the eight lanes of a scale: lane k of them is left with key k's, and works out its scale for all (each lane
    // for each key: 8192 rows 1.0 us more, 24 sequences 0.7)
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) {
      const bool up = (lane & o) != 0;
#pragma unroll
      for (int k = 0; k < o; ++k) {
        const unsigned send = up ? top[k] : top[k + o], stay = up ? top[k + o] : top[k];
        top[k] = max(stay, __shfl_xor_sync(ALL, send, o));
      }
    }
    if (__any_sync(ALL, top[0] >= __float_as_uint(Q4_LARGE))) {
      uint2 v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = x[j];
      uint32_t add[4];
      mine = any_values(v, add);
#pragma unroll
      for (int e = 0; e < 4; ++e) w[i][e] += add[e];
    } else {
      const Q4Scale s = q4_scale(__uint_as_float(top[0] & 0xffff0000u));
      mine = s.code;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float a_scale = __shfl_sync(ALL, s.scale, (lane & 24) | j), its = __shfl_sync(ALL, s.reciprocal, (lane & 24) | j);
        const float2 sc = make_float2(a_scale, a_scale), rc = make_float2(its, its);
        const int2 n0 = q4_whole2(make_float2(bf16lo(x[j].x), bf16hi(x[j].x)), sc, rc);
        const int2 n1 = q4_whole2(make_float2(bf16lo(x[j].y), bf16hi(x[j].y)), sc, rc);
        w[i][0] += (unsigned)n0.x << q4_shift(j);
        w[i][1] += (unsigned)n0.y << q4_shift(j);
        w[i][2] += (unsigned)n1.x << q4_shift(j);
        w[i][3] += (unsigned)n1.y << q4_shift(j);
      }
    }
    const int j = lane & 7;
    if (j >= lo && j < hi) page[Q4_SCALES + (lane >> 3) * 128 + slot + 8 * i + j] = (uint8_t)mine;
    if (i + 1 < WORDS)
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = next[j];
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (WORDS == 4) *reinterpret_cast<uint4*>(words + 4 * e) = make_uint4(w[0][e], w[1][e], w[2][e], w[3][e]);
    else words[4 * e] = w[0][e];
  }
}

// Keys, of eight lanes with a head: a lane's two runs of 8 dims are a word each, four lanes have a scale together.
__device__ __forceinline__ void append_key(const KvAppendQ4Args& a, const Head& h, int g, int page, int slot, int lane,
                                           bool used) {
  unsigned ta = 0, tb = 0;               // (as bits: NaN lies above everything)
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    ta = max(ta, __float_as_uint(h.v[e].x) & 0x7fffffffu);
    tb = max(tb, __float_as_uint(h.v[e].y) & 0x7fffffffu);
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    ta = max(ta, __shfl_xor_sync(ALL, ta, o));
    tb = max(tb, __shfl_xor_sync(ALL, tb, o));
  }
  uint32_t wa = 0x88888888u, wb = 0x88888888u, mine;
  if (__any_sync(ALL, max(ta, tb) >= __float_as_uint(Q4_LARGE))) {
    const float2* v = h.v;
    const uint2 ra = q4_any(make_float4(v[0].x, v[1].x, v[2].x, v[3].x), make_float4(v[4].x, v[5].x, v[6].x, v[7].x), 4);
    const uint2 rb = q4_any(make_float4(v[0].y, v[1].y, v[2].y, v[3].y), make_float4(v[4].y, v[5].y, v[6].y, v[7].y), 4);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      wa += (((ra.x >> (4 * e)) & 15u) - 8u) << q4_shift(e);
      wb += (((rb.x >> (4 * e)) & 15u) - 8u) << q4_shift(e);
    }
    mine = ra.y | (rb.y << 16);
  } else {
    const Q4Scale sa = q4_scale(__uint_as_float(ta)), sb = q4_scale(__uint_as_float(tb));
    const float2 sc = make_float2(sa.scale, sb.scale), rc = make_float2(sa.reciprocal, sb.reciprocal);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int2 n = q4_whole2(h.v[e], sc, rc);
      wa += (unsigned)n.x << q4_shift(e);
      wb += (unsigned)n.y << q4_shift(e);
    }
    mine = sa.code | (sb.code << 16);
  }
  // scales of dims 0, 32, 64, 96 ..: lanes 0 and 4 of the eight
  const unsigned codes = mine | (__shfl_xor_sync(ALL, mine, 4) << 8);
  if (!used) return;
  uint8_t* p = a.Kpool + ((size_t)g * a.num_pages + page) * Q4_BYTES;
  const int l = lane & 7;
  uint32_t* word = reinterpret_cast<uint32_t*>(p + (l >> 2) * Q4_PLANE + slot * 16) + (l & 3);
  word[0] = wa;
  word[2 * Q4_PLANE / 4] = wb;
  if (l == 0) reinterpret_cast<uint32_t*>(p + Q4_SCALES)[slot] = codes;
}

// CTAs: a thread per sequence that checks its bounds (no row has to be in a sequence that breaks them) and blocks of values, a
// warp each, then one CTA per row for its keys and queries.  (8192 rows: without a bound on the registers 44 us, with 12 CTAs an SM 40.7.)
template <int WARPS, int UNITS, int LB>
__global__ void __launch_bounds__(32 * WARPS, WARPS == 2 ? 14 : 5) kv_append_q4_kernel(const KvAppendQ4Args a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, i0 = (lane & 7) * 8;
  if (blockIdx.x < (unsigned)a.check_ctas) {
    check_sequence(a, (long long)blockIdx.x * (32 * WARPS) + threadIdx.x, 0x8F1u);
    return;
  }
  if (blockIdx.x < (unsigned)(a.check_ctas + a.value_ctas)) {
    const unsigned u = (blockIdx.x - a.check_ctas) * WARPS + warp;
    if (u < (unsigned)a.blocks * a.Hkv) append_values<LB>(a, u / a.Hkv, u % a.Hkv, lane);
    return;
  }
  const int r = blockIdx.x - a.check_ctas - a.value_ctas;
  Turns t;
  if (a.cs) t = turns_of(a.cs, r, i0);
  int b = -2, page = 0, p = 0;
  // the row's sequence, position and page, looked up beside the first loads; false: padding
  auto place = [&]() {
    if (b != -2) return b >= 0;
    const Place at = place_of(r, a, lane);
    b = at.b;
    if (b < 0 || r >= at.c1 || out_of_bounds(at.c0, at.c1, at.ctx, a)) {
      b = -1;
      return false;
    }
    p = at.ctx + (r - at.c0);
    page = a.block_table[(size_t)b * a.max_pages + p / Q4_PAGE];
    if (page < 0 || page >= a.num_pages) {
      if (threadIdx.x == 0) set_status(a.status, 0x8F2u);
      page = -1;
    }
    return true;
  };
  each_head<WARPS, 1>(a.Knew + (size_t)r * a.ldkv, a.Hkv, a.wk, a.eps, a.cs != nullptr, t, place, [&](int hd, const Head& h) {
    append_key(a, h, hd, page, p % Q4_PAGE, lane, hd < a.Hkv && page >= 0);
  });
  if (a.Hq > 0 && place())
    each_head<WARPS, UNITS>(a.Q + (size_t)r * a.ldq, a.Hq, a.wq, a.eps, a.cs != nullptr, t, place, [&](int hd, const Head& h) {
      if (hd < a.Hq) store_head(a.Qrot + (size_t)r * a.ldqr + (size_t)hd * D + i0, h);
    });
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
  const Block k = block_of<5>(u / a.Hkv, a, lane);
  if (k.b < 0 || !page_exists(k, a, lane, 0x9F2u)) return;
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
  // (all loads ahead of the stores, which they would otherwise stay behind: 77 keys 5.6 us)
  uint32_t wa[8], wb[8], cs[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int slot = slot0 + 4 * i + (lane >> 3);
    const uint32_t* word = reinterpret_cast<const uint32_t*>(kp + (l >> 2) * Q4_PLANE + slot * 16) + (l & 3);
    wa[i] = word[0];
    wb[i] = word[2 * Q4_PLANE / 4];
    cs[i] = reinterpret_cast<const uint32_t*>(kp + Q4_SCALES)[slot] >> (8 * (l >> 2));
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int j = 4 * i + (lane >> 3);
    if (j < k.lo || j >= k.hi) continue;
    const uint32_t sa = q4_scale2((cs[i] & 255u) * 0x10001u), sb = q4_scale2(((cs[i] >> 16) & 255u) * 0x10001u);
    const uint32_t oa = q4_offset2(sa), ob = q4_offset2(sb);
    uint16_t* dst = a.Kout + (size_t)(k.row0 + j) * a.ldkv + (size_t)g * D + l * 8;
    st_past_l1(dst, make_uint4(q4_pair<0>(wa[i], sa, oa), q4_pair<1>(wa[i], sa, oa), q4_pair<2>(wa[i], sa, oa),
                               q4_pair<3>(wa[i], sa, oa)));
    st_past_l1(dst + 64, make_uint4(q4_pair<0>(wb[i], sb, ob), q4_pair<1>(wb[i], sb, ob), q4_pair<2>(wb[i], sb, ob),
                                    q4_pair<3>(wb[i], sb, ob)));
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

// CTAs of two warps where there are more than four rows for each SM, of four below, where they shorten a row's chain
// (norm with 32 / 8 heads, in us, four warps and two: 8 rows 3.5 / 4.1, 400 4.1 / 4.2, 600 4.8 / 4.8 to 5.5, 900 6.9 / 6.2, 8192
// 37.6 / 29.3; append 8 rows 4.1 / 4.8, 600 5.5 to 8.9 / 6.2 to 8.2, 900 8.6 / 7.6, 8192 57 / 40.6).
cudaError_t launch_qk_norm_rope(const NormRopeArgs& a, int sms, cudaStream_t s) {
  const bool many = a.M > 4 * sms;
  auto* k = many ? qk_norm_rope_kernel<2, 2> : qk_norm_rope_kernel<4, 3>;
  cudaError_t e = launch_k(k, dim3((unsigned)a.M), dim3(many ? 64 : 128), 0, s, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// Values in blocks of 32 keys write whole 16-byte rows of a page, in blocks of 8 a word of each, and leave four times as many
// warps.  The wide ones are taken where sequences bring at least two of them and they alone are ten warps an SM (32 / 8 heads,
// keys and values only, in us, blocks of 8 and of 32: one sequence of 600 rows 3.5 / 9.6, 5000 12.3 / 12.4, 6500 15.0 / 14.3, 8192
// 16.6 / 15.2; with queries and norms 8192 39.0 / 38.6).
cudaError_t launch_kv_append_q4(const KvAppendQ4Args& args, int sms, cudaStream_t s) {
  KvAppendQ4Args a = args;
  const bool many = a.M > 4 * sms, wide = many && a.M >= 64ll * a.B && (long long)(a.M >> 5) * a.Hkv >= 10 * sms;
  const int warps = many ? 2 : 4;
  a.blocks = (a.M >> (wide ? 5 : 3)) + 2 * a.B;
  a.value_ctas = (a.blocks * a.Hkv + warps - 1) / warps;
  a.check_ctas = (a.B + 32 * warps - 1) / (32 * warps);
  auto* k = many ? (wide ? kv_append_q4_kernel<2, 2, 5> : kv_append_q4_kernel<2, 2, 3>)
                 : kv_append_q4_kernel<4, 3, 3>;
  cudaError_t e = launch_k(k, dim3((unsigned)a.M + a.value_ctas + a.check_ctas), dim3(32 * warps), 0, s, a);
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
