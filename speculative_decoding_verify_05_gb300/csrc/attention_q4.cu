// Attention of a few rows per sequence (decode steps, verify rounds) over the paged cache in 4 bits, on tcgen05 tensor
// cores: the R = G * rows <= 64 query rows of a kv head attend their sequence's keys, a page (128 keys) at a time.
//
// Products.  The cache's side is the MMA's 128 rows (its A operand), the queries its N = 16 .. 64 columns:
//   S[key, row] = K . Q^T     M = 128 keys, K = 128 dims
//   O[dim, row] += V^T . P    M = 128 dims, K = 128 keys
// so a tile of 128 x 128 cached values is never padded, however few the rows.  K and V^T go to TMEM, not to shared
// memory: a thread unpacks one row (a key's dims; a dim's keys, which is why the cache holds values transposed) to 64
// registers of bf16 pairs and stores them to its TMEM lane, where the MMA reads its A operand.  Through shared memory the same
// tiles would be written and read again at 128 bytes a cycle: 64 KB in and 64 KB out a page of keys and values, 1024
// cycles, where HBM takes 740 to bring the page.  Only Q and P (bf16, N columns) are read from shared memory.  P is bf16 because
// the MMA takes both operands in one type, and the cache's side is exact in bf16; the sums take the weights before that
// rounding.  It is as large as the output's own: outputs are off by 2.3e-3 of their rms, 1.7e-3 with weights in fp32.
//
// Work.  An item is a (sequence, kv head).  The tiles of all items in a row are cut into equal shares by cost, one for each
// of a CTA's two slots; every slot works its own out from the lengths on the device.  The slots run on their own, each
// with its warps, K, V, S and O tiles in TMEM (4 x 64 columns, all 512 for both) and page rings, so that one goes on while the
// other starts or ends an item (with an item's tiles in turn to both, ending an item cost 4 us of the CTA: 64
// sequences of 2 to 11 rows 126 us).  Pieces of an item that several slots share go to the
// workspace as unnormalised O, reference and sum; the warps of its slots that are done when the last piece arrives join
// it, rows or parts of rows at a time, in order of the slots whoever does it.
//
// Bound.  Not HBM, though the work is a stream of pages: 16 sequences of one token at 30000 keys (32 / 8 heads) take 106
// us = 4.8 TB/s where the copy takes 77, 64 sequences of 2 to 11 rows at up to 8192 keys 98 us of 47.  A page of keys and
// one of values are 32768 entries to unpack, 725 warp instructions for each quarter of the SM with their share of the
// softmax, and a slot's tiles wait for one another: unpack K, score, weigh, and only then P V, whose end frees V's and
// P's place.  The SM issues in 72 % of the cycles with 16 columns, in 58 % with 48, where the softmax's share of
// that chain is three times as long (a tile of a slot takes about 1.2 us with 16 columns, 1.6 with 48).  With few keys to
// a slot: 4 us to the first product (lengths, page table, first pages), 4 to 5 to join shared items; 4 sequences of one token
// at 300 to 1000 keys 11.0 us.  Tried without gain: two places for P, tiles brought to bf16 in halves, eight softmax warps a
// slot, fewer columns for the sequences of few rows in a batch of more.
//
// Roles (28 warps; four to a slot where not said otherwise): 0-7 softmax and epilogue (a thread per key, then per dim); 8 and 9
// issue a slot's MMAs; 10 and 11 walk the batch for a slot, post its pieces and load its queries and pages; 12-19
// bring keys to bf16, 20-27 values.
#include "attention_util.cuh"
#include "internal.h"
#include "q4.cuh"

#include <climits>

namespace spec {
namespace {

constexpr int D = 128;
constexpr int KT = 128;                   // keys per tile (one page)
constexpr int MAXR = 64;                  // rows of an item
constexpr int PR = 4;                     // posted pieces of a slot
constexpr int THREADS = 896;
constexpr int REGS_ALL = 72;
constexpr uint32_t TMEM_COLS = 512, T_K = 0, T_V = 128, T_S = 256, T_O = 384;   // 64 columns for each slot

constexpr uint64_t JOIN_WAIT_NS = 20000;  // how long a warp that is done waits for the other pieces of a shared item
// What an item's start and end cost, in keys (64 sequences of 2 to 11 rows: 98.2 us, with 160 104.8, with 640 100.4).
constexpr int ITEM_KEYS = 320;
// What a piece costs the join, in keys (see shares_of): one sequence of one kv head, 8 query heads, at 20000 keys 13.0 us, at
// 1000 8.9; cut into equal shares down to single tiles 17.8 and 13.4, with 1 key a piece 14.5 and 9.2.
constexpr int PIECE_KEYS = 3;

__device__ __forceinline__ void bar_sync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }
__device__ __forceinline__ bool bar_or(int id, int n, bool x) {
  uint32_t r;
  asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, %2, %3, p;\n selp.u32 %0, 1, 0, q;\n}"
               : "=r"(r)
               : "r"((uint32_t)x), "r"(id), "r"(n)
               : "memory");
  return r != 0;
}
// Columns folded over a warp's lanes: v[0] of lane i is then column i mod 16 of all 32 lanes.  Each step halves the columns
// that a lane still holds (16 shuffles; a reduction instruction per column took longer than all of a tile's weights).
template <class F>
__device__ __forceinline__ void fold16(float (&v)[16], int lane, F&& f) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float send = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
      v[i] = f(keep, __shfl_xor_sync(0xffffffffu, send, o));
    }
  }
  v[0] = f(v[0], __shfl_xor_sync(0xffffffffu, v[0], 16));
}
template <int N>
struct Int {
  static constexpr int value = N;
};

// ----------------------------------------------------------------- the batch
struct Seq {
  int r0, rows, ctx;
};
// Sequence b; one that breaks its bounds counts as having no rows (*bad set).
__device__ __forceinline__ Seq seq_of(const ChunkAttnArgs& a, int b, bool* bad = nullptr) {
  const int c0 = a.cu_rows[b], c1 = a.cu_rows[b + 1], ctx = a.ctx_len[b];
  const bool ok = c0 >= 0 && c1 >= c0 && c1 <= a.M && c1 - c0 <= a.max_rows &&
                  (c0 == c1 || (ctx >= 0 && (long long)ctx + (c1 - c0) <= (long long)a.max_pages * KT));
  if (bad) *bad = !ok;
  return Seq{c0, ok ? c1 - c0 : 0, ctx};
}
__device__ __forceinline__ long long item_cost(const Seq& s) { return (long long)s.ctx + s.rows + ITEM_KEYS; }
// The tile that a cut at cost y of an item (its start 0) falls before: 0 .. nt.
__device__ __forceinline__ int cut_tile(long long y, int keys, int nt) {
  y -= ITEM_KEYS;
  if (y <= 0) return 0;
  if (y >= keys) return nt;
  const int t = ((int)y + KT / 2) / KT;
  return t * KT + KT / 2 >= keys ? nt : t;              // (no piece of a few keys)
}
// The cost of the batch and of a slot's share of it.  Equal shares, but of so many keys that an item's pieces are not
// joined for longer than they take.
struct Shares {
  long long total, each;
  __device__ __forceinline__ long long start(int c) const { return min(total, c * each); }
};
__device__ __forceinline__ Shares shares_of(const ChunkAttnArgs& a, long long total, int keys) {
  const long long even = (long long)__umul64hi((unsigned long long)total, a.inv_grid) / 2 + 1;      // (two slots)
  return Shares{total, max(even, (long long)sqrtf((float)PIECE_KEYS * keys))};
}

// A slot's consecutive tiles of one item, as posted.
struct Piece {
  int b, h;
  int t0, t1, nt;      // tiles t0 .. t1 - 1 of the item's nt
  int row0, rows, ctx;
  int more;            // 0: no piece, the slot is done
  long long start;     // cost of everything before the item
  __device__ __forceinline__ int tiles() const { return t1 - t0; }
  __device__ __forceinline__ bool shared() const { return t0 > 0 || t1 < nt; }
};

// NC: columns of the MMAs (rows of the queries, a multiple of 16).
template <int NC>
struct Layout {
  // Registers: of few columns the softmax leaves some to the warps that bring pages to bf16 (16 x 1 row at 30000 keys
  // 112.9 us with the other split).
  static constexpr int REGS_SOFTMAX = NC <= 16 ? 96 : 112, REGS_ROLES = 56, REGS_BF16 = NC <= 16 ? 64 : 56;
  static_assert(256 * REGS_SOFTMAX + 128 * REGS_ROLES + 512 * REGS_BF16 <= THREADS * REGS_ALL, "register split");
  // Pages in flight of a slot, of keys and of values (64 sequences of 2 to 11 rows, in 48 columns: 100.1 us with 3)
  static constexpr int SP = NC <= 48 ? 4 : 3;
  static constexpr int Q_HALF = NC * 128;                         // rows x 64 dims (128-byte swizzled rows)
  static constexpr int OFF_P = 0;                                 // of each slot: [key][row], 128-byte swizzled rows
  static constexpr int OFF_Q = OFF_P + 2 * KT * 128;              // of each slot two buffers of two halves
  static constexpr int OFF_KP = OFF_Q + 2 * 2 * 2 * Q_HALF;
  static constexpr int OFF_VP = OFF_KP + 2 * SP * Q4_BYTES;
  static constexpr int OFF_EXP = OFF_VP + 2 * SP * Q4_BYTES;      // scales of a tile of values, as pairs
  static constexpr int OFF_REF = OFF_EXP + 4096;                  // [2][64] references
  static constexpr int OFF_ADD = OFF_REF + 2 * MAXR * 4;          // [2][64] what is added to a score for it
  static constexpr int OFF_ALPHA = OFF_ADD + 2 * MAXR * 4;        // [2][64] factors (of an end: what O is multiplied by)
  static constexpr int OFF_MAX = OFF_ALPHA + 2 * MAXR * 4;        // [8][64] maxima, later sums, of the softmax warps
  static constexpr int OFF_TOK = OFF_MAX + 8 * MAXR * 4;          // [64] token of each row
  static constexpr int OFF_PIECE = OFF_TOK + MAXR * 4;            // [2][PR + 1]: posted, and the slot's first for the end
  static constexpr int OFF_SHARES = OFF_PIECE + 2 * (PR + 1) * (int)sizeof(Piece);
  static constexpr int OFF_BAR = OFF_SHARES + 2 * (int)sizeof(Shares);
  static constexpr int N_BARS = 2 * (4 * SP + 6 + 4 + 2 * PR);
  static constexpr int OFF_MORE = OFF_BAR + N_BARS * 8;           // marks of the page rings' stages, then the TMEM address
  static constexpr int SMEM = OFF_MORE + 2 * 2 * SP * 4 + 8;
  static_assert(OFF_KP % 128 == 0 && OFF_EXP % 16 == 0 && OFF_PIECE % 8 == 0 && OFF_BAR % 8 == 0, "alignment");
  static_assert(SMEM <= 227 * 1024, "shared memory budget");
};

template <int NC>
__global__ void __launch_bounds__(THREADS, 1)
few_attention_q4_kernel(const __grid_constant__ CUtensorMap tmQ, const ChunkAttnArgs a) {
  using L = Layout<NC>;
  constexpr int SP = L::SP;
  extern __shared__ __align__(1024) uint8_t smem[];
  struct Bars {
    uint64_t k_land[SP], k_free[SP];     // page of keys landed, read
    uint64_t v_land[SP], v_free[SP];
    uint64_t ka_full, va_full;           // K, V tile in TMEM
    uint64_t s_full;                     // scores in TMEM (K read)
    uint64_t s_free;                     // ... read
    uint64_t p_full;                     // P in shared memory, O rescaled
    uint64_t o_done;                     // P V done (V and P read, O whole)
    uint64_t q_full[2], q_free[2];
    uint64_t posted[PR], taken[PR];
  };
  static_assert(2 * sizeof(Bars) == L::N_BARS * 8, "barriers");
  Bars* all_bars = reinterpret_cast<Bars*>(smem + L::OFF_BAR);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_MORE + 2 * 2 * SP * 4);
  int* s_tok = reinterpret_cast<int*>(smem + L::OFF_TOK);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if ((smem_u32(smem) & 1023u) != 0) {     // (the swizzled tiles need it; the same for every thread)
    if (tid == 0) set_status(a.status, 0xAF3u);
    return;
  }
  if (tid == 0) {
    tma_prefetch_desc(&tmQ);
    for (int x = 0; x < 2; ++x) {
      Bars& b = all_bars[x];
      for (int i = 0; i < SP; ++i) {
        mbar_init(&b.k_land[i], 1);
        mbar_init(&b.k_free[i], 4);
        mbar_init(&b.v_land[i], 1);
        mbar_init(&b.v_free[i], 4);
      }
      mbar_init(&b.ka_full, 4);
      mbar_init(&b.va_full, 4);
      mbar_init(&b.s_full, 1);
      mbar_init(&b.s_free, 4);
      mbar_init(&b.p_full, 4);
      mbar_init(&b.o_done, 1);
      for (int i = 0; i < 2; ++i) {
        mbar_init(&b.q_full[i], 1);
        mbar_init(&b.q_free[i], 1);
      }
      for (int i = 0; i < PR; ++i) {
        mbar_init(&b.posted[i], 1);
        mbar_init(&b.taken[i], 5);         // MMA, 4 softmax warps
      }
    }
    fence_barrier_init();
  }
  if (tid < MAXR) s_tok[tid] = tid / a.G;
  if (warp == 8) tmem_alloc(tmem_slot, TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (*tmem_slot != 0 && tid == 0) set_status(a.status, 0xAF4u);       // (all 512 columns are this CTA's)
  // everything above overlaps the kernel before; global memory only below
  pdl_wait();
  pdl_trigger();

  // slot of the warp: softmax 0-7, MMA 8 and 9, pages 10 and 11, keys 12-19, values 20-27
  const int slot = warp < 8 || warp >= 12 ? (warp >> 2) + (warp >= 12 ? 1 : 0) & 1 : warp & 1;
  Bars& bar = all_bars[slot];
  Piece* ring = reinterpret_cast<Piece*>(smem + L::OFF_PIECE) + slot * (PR + 1);
  Piece* s_first = ring + PR;
  Shares* s_shares = reinterpret_cast<Shares*>(smem + L::OFF_SHARES) + slot;
  int* k_more = reinterpret_cast<int*>(smem + L::OFF_MORE) + slot * 2 * SP;      // [SP] 0: nothing more from this stage on
  int* v_more = k_more + SP;
  const int me = blockIdx.x * 2 + slot;

  if (warp >= 12) {
    // -------------------------------------------------------------- pages to bf16: keys (12-19), values (20-27)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(L::REGS_BF16));
    const bool is_v = warp >= 20;
    const int row = tid & 127;
    const uint32_t t_dst = (is_v ? T_V : T_K) + slot * 64 + (uint32_t((warp & 3) * 32) << 16);
    uint64_t *land = is_v ? bar.v_land : bar.k_land, *free_ = is_v ? bar.v_free : bar.k_free;
    uint64_t *full = is_v ? &bar.va_full : &bar.ka_full, *gone = is_v ? &bar.o_done : &bar.s_full;
    const int* more = is_v ? v_more : k_more;
    uint4* exp = reinterpret_cast<uint4*>(smem + L::OFF_EXP) + (warp & 7) * 32;
    bool ok = true;
    for (int n = 0;; ++n) {
      const int st = n % SP;
      ok = __all_sync(0xffffffffu, wait_for(&land[st], (uint32_t)((n / SP) & 1)));
      if (!ok || !more[st]) break;
      const uint8_t* page = smem + (is_v ? L::OFF_VP : L::OFF_KP) + (slot * SP + st) * Q4_BYTES;
      uint4 w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) w[q] = *reinterpret_cast<const uint4*>(page + q * Q4_PLANE + row * 16);
      // keys: their own four scales; values: those of the 4 keys whose scales this lane spreads for the warp
      const uint32_t codes = *reinterpret_cast<const uint32_t*>(page + Q4_SCALES + row * 4);
      if (is_v) {
        const uint32_t c0 = __byte_perm(codes, 0, 0x4140), c1 = __byte_perm(codes, 0, 0x4342);
        exp[lane] = make_uint4(q4_even2(c0), q4_less2(c0), q4_odd2(c1), q4_less2(c1));
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&free_[st]);
      if (n > 0) ok = wait_for(gone, (uint32_t)((n - 1) & 1));
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t r[16];
        const uint32_t x[4] = {w[q].x, w[q].y, w[q].z, w[q].w};
        if (!is_v) {
          const uint32_t c = __byte_perm(codes, 0, 0x4040 | q * 0x0101);
          const uint32_t even = q4_even2(c), odd = q4_odd2(c), less = q4_less2(c);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t x8 = x[i] >> 8;
            r[4 * i] = q4_tile_pair<0>(x[i], x8, even, less);
            r[4 * i + 1] = q4_tile_pair<1>(x[i], x8, odd, less);
            r[4 * i + 2] = q4_tile_pair<2>(x[i], x8, even, less);
            r[4 * i + 3] = q4_tile_pair<3>(x[i], x8, odd, less);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 e0 = exp[8 * q + 2 * i], e1 = exp[8 * q + 2 * i + 1];
            const uint32_t x8 = x[i] >> 8;
            r[4 * i] = q4_tile_pair<0>(x[i], x8, e0.x, e0.y);
            r[4 * i + 1] = q4_tile_pair<1>(x[i], x8, e0.z, e0.w);
            r[4 * i + 2] = q4_tile_pair<2>(x[i], x8, e1.x, e1.y);
            r[4 * i + 3] = q4_tile_pair<3>(x[i], x8, e1.z, e1.w);
          }
        }
        tmem_st_cols16(t_dst + q * 16, r);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(full);
    }
    if (!ok) set_status(a.status, 0x851u);
  } else if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(L::REGS_ROLES));
    if (warp >= 10) {
      // ------------------------------------------------------------ pieces, queries, pages
      const int run = (a.B + 31) >> 5, b0 = min(lane * run, a.B), b1 = min(b0 + run, a.B);
      long long own = 0;
      bool bad = false;
      int longest = 0;
#pragma unroll 4
      for (int b = b0; b < b1; ++b) {
        bool wrong;
        const Seq s = seq_of(a, b, &wrong);
        bad |= wrong;
        if (s.rows > 0) {
          own += item_cost(s) * a.Hkv;
          longest = max(longest, s.ctx + s.rows);
        }
      }
      if (bad && me == 0) set_status(a.status, 0xAF1u);
      long long before = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += v;
      }
      const Shares shares = shares_of(a, __shfl_sync(0xffffffffu, before, 31),
                                      (int)__reduce_max_sync(0xffffffffu, (unsigned)longest));
      before -= own;
      // where a cut falls: before tile t of kv head h of sequence b
      struct Cut {
        int b, h, t;
        Seq s;
        long long start;
      };
      auto cut_at = [&](long long x) {
        Cut c{a.B, 0, 0, Seq{0, 0, 0}, 0};
        const unsigned owner = __ballot_sync(0xffffffffu, x >= before && x < before + own);
        if (owner == 0) return c;              // (the end of everything, or nothing at all)
        long long at = before;
        if (x >= before && x < before + own)
          for (c.b = b0;; ++c.b) {
            c.s = seq_of(a, c.b);
            const long long all = c.s.rows > 0 ? item_cost(c.s) * a.Hkv : 0;
            if (x < at + all) break;
            at += all;
          }
        const int from = __ffs(owner) - 1;
        c.b = __shfl_sync(0xffffffffu, c.b, from);
        c.s.r0 = __shfl_sync(0xffffffffu, c.s.r0, from);
        c.s.rows = __shfl_sync(0xffffffffu, c.s.rows, from);
        c.s.ctx = __shfl_sync(0xffffffffu, c.s.ctx, from);
        at = __shfl_sync(0xffffffffu, at, from);
        const long long item = item_cost(c.s);
        c.h = (int)((unsigned long long)(x - at) / (unsigned long long)item);
        c.start = at + c.h * item;
        const int keys = c.s.ctx + c.s.rows;
        c.t = cut_tile(x - c.start, keys, (keys + KT - 1) / KT);
        return c;
      };
      Cut c = cut_at(shares.start(me));
      const Cut e = cut_at(shares.start(me + 1));
      const uint64_t pol = l2_policy_evict_first();
      const uint32_t q_bytes = (uint32_t)(a.tpt * a.G * D * 2);
      bool ok = true;
      int n = 0, k = 0;                      // tiles and pieces so far
      auto stage_free = [&](int n) {
        const int st = n % SP;
        if (n >= SP)
          ok = ok && wait_for(&bar.k_free[st], (uint32_t)((n / SP - 1) & 1)) &&
               wait_for(&bar.v_free[st], (uint32_t)((n / SP - 1) & 1));
        ok = __all_sync(0xffffffffu, ok);
        return st;
      };
      for (;;) {
        Piece p{};
        if (c.b < a.B) {
          const int keys = c.s.ctx + c.s.rows;
          p = Piece{c.b, c.h, c.t, (keys + KT - 1) / KT, (keys + KT - 1) / KT, c.s.r0, c.s.rows, c.s.ctx, 1, c.start};
          const bool last = c.b == e.b && c.h == e.h;
          if (last) p.t1 = e.t;
          if (c.b > e.b || (c.b == e.b && c.h > e.h)) p.more = 0;
          else if (p.t1 <= p.t0) p.more = last ? 0 : -1;             // (nothing of this item)
        }
        if (p.more >= 0) {
          ok = __all_sync(0xffffffffu, ok && (k < PR || wait_for(&bar.taken[k % PR], (uint32_t)((k / PR - 1) & 1))));
          if (!ok) break;
          if (lane == 0) {
            if (k == 0) {
              *s_first = p;
              *s_shares = shares;
            }
            ring[k % PR] = p;
            mbar_arrive(&bar.posted[k % PR]);
          }
          __syncwarp();
          if (p.more == 0) break;
          const int qb = k & 1;
          if (k >= 2) ok = wait_for(&bar.q_free[qb], (uint32_t)(((k >> 1) - 1) & 1));
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (lane == 0) {
            uint8_t* dst = smem + L::OFF_Q + (slot * 2 + qb) * 2 * L::Q_HALF;
            mbar_arrive_expect_tx(&bar.q_full[qb], q_bytes);
            tma_load_3d(dst, &tmQ, &bar.q_full[qb], 0, p.h * a.G, p.row0);
            tma_load_3d(dst + L::Q_HALF, &tmQ, &bar.q_full[qb], 64, p.h * a.G, p.row0);
          }
          ++k;
          int ids = 0, base = -1;            // page ids of 32 tiles at a time, one per lane
          for (int t = p.t0; t < p.t1; ++t, ++n) {
            if (base < 0 || t >= base + 32) {
              base = t;
              ids = t + lane < p.t1 ? a.block_table[(size_t)p.b * a.max_pages + t + lane] : 0;
              if (ids < 0 || ids >= a.num_pages) {
                set_status(a.status, 0xAF2u);
                ids = 0;
              }
            }
            const size_t at = ((size_t)p.h * a.num_pages + __shfl_sync(0xffffffffu, ids, t - base)) * Q4_BYTES;
            const int st = stage_free(n);
            if (!ok) break;
            if (lane == 0) {
              uint8_t *kd = smem + L::OFF_KP + (slot * SP + st) * Q4_BYTES, *vd = smem + L::OFF_VP + (slot * SP + st) * Q4_BYTES;
              k_more[st] = v_more[st] = 1;
              mbar_arrive_expect_tx(&bar.k_land[st], Q4_BYTES);
              bulk_load_hint(kd, static_cast<const uint8_t*>(a.Kpool) + at, Q4_BYTES, &bar.k_land[st], pol);
              mbar_arrive_expect_tx(&bar.v_land[st], Q4_BYTES);
              bulk_load_hint(vd, static_cast<const uint8_t*>(a.Vpool) + at, Q4_BYTES, &bar.v_land[st], pol);
            }
          }
          if (!ok) break;
        }
        // the next item
        c.t = 0;
        c.start += item_cost(c.s);
        if (++c.h == a.Hkv) {
          c.h = 0;
          // the next sequence with rows, 32 candidates at a time (a padded batch may have hundreds without)
          int from = c.b + 1;
          for (c.b = a.B; from < a.B && from <= e.b; from += 32) {
            const Seq s = from + lane < a.B ? seq_of(a, from + lane) : Seq{0, 0, 0};
            const unsigned has = __ballot_sync(0xffffffffu, s.rows > 0);
            if (has == 0) continue;
            const int i = __ffs(has) - 1;
            c.b = from + i;
            c.s.r0 = __shfl_sync(0xffffffffu, s.r0, i);
            c.s.rows = __shfl_sync(0xffffffffu, s.rows, i);
            c.s.ctx = __shfl_sync(0xffffffffu, s.ctx, i);
            break;
          }
        }
      }
      const int loads = n;
      if (ok) {                              // nothing more to bring to bf16
        const int st = stage_free(n);
        if (ok && lane == 0) {
          k_more[st] = v_more[st] = 0;
          mbar_arrive(&bar.k_land[st]);
          mbar_arrive(&bar.v_land[st]);
        }
      }
      if (!ok) {                             // gave up: see the copies in flight land before leaving
        set_status(a.status, 0x811u);
        for (int j = loads > SP ? loads - SP : 0; j < loads; ++j) {
          wait_for(&bar.k_land[j % SP], (uint32_t)((j / SP) & 1));
          wait_for(&bar.v_land[j % SP], (uint32_t)((j / SP) & 1));
        }
        for (int j = k > 2 ? k - 2 : 0; j < k; ++j) wait_for(&bar.q_full[j & 1], (uint32_t)((j >> 1) & 1));
      }
      __syncwarp();
    } else {
      // ------------------------------------------------------------ MMA issue
      // A tile's scores are issued as soon as the softmax has those before them in its registers, while it works on them and
      // ahead of their P V.  The whole warp walks the tiles and one elected
      // lane issues; after a wait that ran out it goes on without waiting (to garbage that nobody reads).
      const bool leader = elect_one();
      constexpr uint32_t idesc_s = umma_idesc_bf16(KT, NC), idesc_pv = umma_idesc_bf16(D, NC) | (1u << 16);   // (P: MN-major)
      const uint32_t t0 = slot * 64;
      bool ok = true;
      auto wait = [&](uint64_t* b, uint32_t parity) {
        if (ok) ok = wait_for(b, parity);
      };
      struct Cursor {
        int k, j, tiles, more;               // piece, its tile, tiles
      };
      auto enter = [&](Cursor& c) {
        wait(&bar.posted[c.k % PR], (uint32_t)((c.k / PR) & 1));
        ok = __all_sync(0xffffffffu, ok);
        const Piece& p = ring[c.k % PR];
        c.j = 0;
        c.tiles = p.tiles();
        c.more = ok && p.more;
      };
      auto step = [&](Cursor& c) {
        if (++c.j == c.tiles) {
          ++c.k;
          enter(c);
        }
      };
      auto scores = [&](int n, Cursor& c) {
        const int qb = c.k & 1;
        if (c.j == 0) wait(&bar.q_full[qb], (uint32_t)((c.k >> 1) & 1));
        wait(&bar.ka_full, (uint32_t)(n & 1));
        tc_fence_after();
        if (leader) {
          const uint64_t qd = umma_desc_sw128(smem_u32(smem + L::OFF_Q + (slot * 2 + qb) * 2 * L::Q_HALF));
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_bf16_ts(T_S + t0, T_K + t0 + kk * 8, qd + (((kk >> 2) * L::Q_HALF + (kk & 3) * 32) >> 4), idesc_s,
                         kk > 0 ? 1u : 0u);
          umma_commit(&bar.s_full);
          if (c.j + 1 == c.tiles) umma_commit(&bar.q_free[qb]);
        }
        __syncwarp();
      };
      Cursor cs{0, 0, 0, 0}, cp{0, 0, 0, 0};
      enter(cs);
      cp = cs;
      if (cs.more) {
        scores(0, cs);
        step(cs);
      }
      for (int n = 0; cp.more; ++n) {
        wait(&bar.s_free, (uint32_t)(n & 1));
        if (cs.more) {
          scores(n + 1, cs);
          step(cs);
        }
        wait(&bar.va_full, (uint32_t)(n & 1));
        wait(&bar.p_full, (uint32_t)(n & 1));
        tc_fence_after();
        if (leader) {
          const uint64_t pd = desc_mn(smem_u32(smem + L::OFF_P + slot * KT * 128), 0);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_bf16_ts(T_O + t0, T_V + t0 + kk * 8, pd + kk * 128, idesc_pv, cp.j > 0 || kk > 0 ? 1u : 0u);
          umma_commit(&bar.o_done);
        }
        __syncwarp();
        const int done = cp.k;
        step(cp);
        if (cp.k != done && lane == 0) mbar_arrive(&bar.taken[done % PR]);
      }
      if (!ok) set_status(a.status, 0x821u);
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(L::REGS_SOFTMAX));
    // ------------------------------------------------------------ softmax and epilogue
    // (After a wait that ran out a warp stops waiting, but keeps the control flow up to the next piece, so that the
    // named barriers stay matched.)
    const int t = tid & 127;               // key of the tile; dim of the output
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    const uint32_t t_s = T_S + slot * 64 + lanes, t_o = T_O + slot * 64 + lanes;
    float* ref = reinterpret_cast<float*>(smem + L::OFF_REF) + slot * MAXR;
    float* add = reinterpret_cast<float*>(smem + L::OFF_ADD) + slot * MAXR;
    float* alpha = reinterpret_cast<float*>(smem + L::OFF_ALPHA) + slot * MAXR;
    float* s_max = reinterpret_cast<float*>(smem + L::OFF_MAX) + slot * 4 * MAXR;
    uint8_t* tile_p = smem + L::OFF_P + slot * KT * 128;
    uint8_t* prow = tile_p + t * 128;
    const float scale = a.scale_log2;
    const int wq = warp & 3;
    bool ok = true;
    uint32_t n = 0;                        // tiles so far
    Shares shares{0, 0};
    const Piece* shared_last = nullptr;    // the slot's last piece, where its item goes on in the next slot
    bool shared_first = false;             // the first piece's item came from the slot before
    // the last slot up to this one whose share does not start inside the item, 32 at a time
    auto first_of = [&](const Piece& p) {
      const int keys = p.ctx + p.rows;
      int c = me;
      for (unsigned out = 0; out == 0; c -= out ? __ffs(out) - 1 : 32)
        out = __ballot_sync(0xffffffffu, cut_tile(shares.start(max(c - lane, 0)) - p.start, keys, p.nt) == 0);
      return c;
    };
    for (int k = 0;; ++k) {
      ok = ok && wait_for(&bar.posted[k % PR], (uint32_t)((k / PR) & 1));
      // (also: everybody has read what the piece before left in shared memory and TMEM)
      if (bar_or(1 + slot, 128, !ok)) {
        ok = false;
        break;
      }
      const Piece& p = ring[k % PR];
      if (k == 0) shares = *s_shares;
      if (!p.more) break;
      const int tiles = p.tiles();
      float2 l[NC / 2];
#pragma unroll
      for (int c = 0; c < NC / 2; ++c) l[c] = make_float2(0.f, 0.f);
      // (columns behind the rows hold anything: their weights are 0, or NaN, and nobody looks at them)
      const int R = p.rows * a.G;
      if (t < MAXR) {
        ref[t] = -INFINITY;
        add[t] = t < R ? 0.f : -INFINITY;
      }
      for (int j = 0; j < tiles; ++j, ++n) {
        const int key = (p.t0 + j) * KT + t;
        const bool masked = (p.t0 + j) * KT + KT - 1 > p.ctx;       // (some row does not see some key)
        ok = ok && wait_for(&bar.s_full, n & 1);
        __syncwarp();
        tc_fence_after();
        // hidden scores become -inf in place (once or twice an item: a loop, so that few instructions are fetched for it)
        if (masked) {
#pragma unroll 1
          for (int c0 = 0; c0 < NC; c0 += 16) {
            uint32_t h[16];
            tmem_ld_cols16(t_s + c0, h);
#pragma unroll
            for (int c = 0; c < 16; ++c)
              if (key > p.ctx + s_tok[c0 + c]) h[c] = 0xff800000u;        // -inf
            tmem_st_cols16(t_s + c0, h);
          }
          tmem_st_wait();
        }
        // Of few columns a thread takes its scores to registers, so that the next tile's can take their place while it works
        // on these (16 x 1 row at 30000 keys 109 -> 105.6 us); 32 and more do not fit beside their sums.
        constexpr bool EARLY = NC <= 16;
        float all[EARLY ? NC : 1];
        auto s_read = [&]() {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.s_free);
        };
        if constexpr (EARLY) {
          tmem_ld_cols<NC>(t_s, all);
          s_read();
        }
        auto get = [&](int c0, float (&x)[16]) {
          if constexpr (EARLY) {
#pragma unroll
            for (int c = 0; c < 16; ++c) x[c] = all[c0 + c];
          } else {
            tmem_ld16(t_s + c0, x);
          }
        };
        // ... as weights: 2 columns from c0 + c
        auto weight = [&](const float (&x)[16], int c0, int c) {
          const float2 r = *reinterpret_cast<const float2*>(add + c0 + c);
          float2 e = fma2(make_float2(x[c], x[c + 1]), make_float2(scale, scale), r);
          e.x = ex2(e.x);
          e.y = ex2(e.y);
          return e;
        };
        // Weights are relative to the row's reference: the maximum of the piece's first tile in which it sees a key, whose
        // own weight is then 1.  Later tiles keep it as long as no weight passes 2^24 (any reference far below
        // the maximum gives the same quotients: bf16 and fp32 have exponents to spare); then the maximum is taken, O and
        // the sums rescaled, and the weights formed again.  (A row that sees no key of the piece's first tile sees none
        // of its later ones.)
        for (bool look = j == 0;; look = true) {
          if (look) {
#pragma unroll
            for (int c0 = 0; c0 < NC; c0 += 16) {
              float x[16];
              get(c0, x);
              fold16(x, lane, [](float a, float b) { return fmaxf(a, b); });
              if (lane < 16) s_max[wq * MAXR + c0 + lane] = x[0];
            }
            bar_sync(1 + slot, 128);
            bool moved = false;
            if (t < R) {
              const float* m4 = s_max + t;
              const float mx = fmaxf(fmaxf(m4[0], m4[MAXR]), fmaxf(m4[2 * MAXR], m4[3 * MAXR])) * scale;
              const float old = ref[t];
              const bool move = old == -INFINITY ? mx > -INFINITY : mx > old + 19.f;
              const float f = move && old != -INFINITY ? ex2(old - mx) : 1.f;
              if (move) {
                ref[t] = mx;
                add[t] = -mx;
              }
              alpha[t] = f;
              moved = f != 1.f;
            }
            if (bar_or(1 + slot, 128, moved)) {
#pragma unroll
              for (int c = 0; c < NC; c += 2) {
                const float2 f = *reinterpret_cast<const float2*>(alpha + c);
                l[c / 2].x *= f.x;
                l[c / 2].y *= f.y;
              }
              ok = ok && wait_for(&bar.o_done, (n - 1) & 1);       // O whole (some tile was before: a factor is not 1)
              __syncwarp();
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < NC; c += 16) {
                uint32_t o[16];
                tmem_ld_cols16(t_o + c, o);
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha[c + i]);
                tmem_st_cols16(t_o + c, o);
              }
              tmem_st_wait();
            }
          }
          if (j > 0) ok = ok && wait_for(&bar.o_done, (n - 1) & 1);      // P read
          uint32_t top = 0;                  // the largest weights of the even and odd columns (NaN is passed over)
#pragma unroll
          for (int c0 = 0; c0 < NC; c0 += 16) {
            float x[16];
            get(c0, x);
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float2 e = weight(x, c0, 2 * i);
              l[c0 / 2 + i] = add2(l[c0 / 2 + i], e);
              w[i] = cvt_bf16x2(e.x, e.y);
              asm("max.bf16x2 %0, %0, %1;" : "+r"(top) : "r"(w[i]));
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
              *reinterpret_cast<uint4*>(prow + ((((c0 >> 3) + i) ^ (t & 7)) << 4)) =
                  make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
          }
          // (0x4B80: 2^24; weights are not negative, so their bits are in order)
          if (look || !bar_or(1 + slot, 128, (top & 0xffffu) > 0x4B80u || (top >> 16) > 0x4B80u)) break;
          // Taken back: what is lost of the sums is 2^-24 of the weights taken back, of which the new reference leaves
          // at most 1 in a sum that has a 1; an infinite one leaves nothing of what was there before.
#pragma unroll
          for (int c0 = 0; c0 < NC; c0 += 16) {
            float x[16];
            get(c0, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float2 e = weight(x, c0, 2 * i);
              float2& s = l[c0 / 2 + i];
              s.x = e.x == INFINITY ? 0.f : s.x - e.x;
              s.y = e.y == INFINITY ? 0.f : s.y - e.y;
            }
          }
        }
        if constexpr (!EARLY) s_read();
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.p_full);
      }
      // ---------------------------------------------------------- end of the piece
      // sums of the warp's 32 keys
      float* sums = s_max + wq * MAXR;
#pragma unroll
      for (int c0 = 0; c0 < NC; c0 += 16) {
        float v[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[2 * i] = l[c0 / 2 + i].x;
          v[2 * i + 1] = l[c0 / 2 + i].y;
        }
        fold16(v, lane, [](float a, float b) { return a + b; });
        if (lane < 16) sums[c0 + lane] = v[0];
      }
      const bool shared = p.shared();
      const int c_first = shared ? first_of(p) : me;
      const size_t at = (size_t)me * 2 + (me == c_first ? 1 : 0);
      bar_sync(1 + slot, 128);
      if (t < R) {
        const float sum = (s_max[t] + s_max[MAXR + t]) + (s_max[2 * MAXR + t] + s_max[3 * MAXR + t]);
        if (shared) __stcg(a.part_ml + at * MAXR + t, make_float2(ref[t], sum));
        else alpha[t] = Q4_TILE_SCALE / sum;
      }
      ok = ok && wait_for(&bar.o_done, (n - 1) & 1);
      bar_sync(1 + slot, 128);
      tc_fence_after();
      // O^T: a dim per thread.  To the workspace as it is; as outputs by way of P's memory, whose rows then leave in
      // 16 bytes a thread.
      uint16_t* rows = reinterpret_cast<uint16_t*>(tile_p);            // [row][dim]
#pragma unroll 1
      for (int c0 = 0; c0 < R; c0 += 16) {
        float o[16];
        tmem_ld16(t_o + c0, o);
        if (shared) {
          float* dst = a.part_o + (at * MAXR + c0) * D + t;
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (c0 + i < R) __stcg(dst + i * D, o[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) rows[(c0 + i) * D + t] = f2bf(o[i] * alpha[c0 + i]);
        }
      }
      tc_fence_before();
      if (shared) {
        if (p.t0 > 0) shared_first = true;
        else shared_last = &p;             // (its entry of the ring is not posted again)
        __syncwarp();
        if (lane == 0) red_release(a.counters + 8 * c_first, (unsigned)tiles);
      } else {
        bar_sync(1 + slot, 128);
        uint16_t* out = a.O + (size_t)p.row0 * a.ldo + (size_t)p.h * a.G * D + (t & 15) * 8;
#pragma unroll 1
        for (int r = t >> 4; r < R; r += 8) {
          const int tok = s_tok[r], g = r - tok * a.G;
          *reinterpret_cast<uint4*>(out + (size_t)tok * a.ldo + g * D) =
              *reinterpret_cast<const uint4*>(rows + r * D + (t & 15) * 8);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.taken[k % PR]);
    }
    if (!ok) set_status(a.status, 0x841u);
    // At the slot's end: the rows of a shared item are joined by the warps of all its slots that are still here when
    // the last piece arrives, a row at a time.  A warp waits for that a while only: the warp that brings the last
    // piece joins whatever is left, so no CTA needs another one to run beside it.
    ok = __all_sync(0xffffffffu, ok);
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      if (!ok || !(i ? shared_first : shared_last != nullptr)) continue;
      const Piece& p = i ? *s_first : *shared_last;
      const int c_first = first_of(p), keys = p.ctx + p.rows, R = p.rows * a.G;
      unsigned *arrived = a.counters + 8 * c_first, *tickets = arrived + 4;
      // the slots that have a piece: those of 32 from `base` on, and the tiles up to the last of them
      struct Sharers {
        unsigned has;
        int t;
      };
      auto sharers = [&](int base, int before) {
        const int to = cut_tile(shares.start(base + lane + 1) - p.start, keys, p.nt);
        const int prev = __shfl_up_sync(0xffffffffu, to, 1);
        return Sharers{__ballot_sync(0xffffffffu, to > (lane == 0 ? before : prev)), __shfl_sync(0xffffffffu, to, 31)};
      };
      const Sharers all = sharers(c_first, 0);
      int count = __popc(all.has);
      Sharers s = all;
      for (int base = c_first; s.t < p.nt; count += __popc(s.has)) s = sharers(base += 32, s.t);
      unsigned there = 0;
      if (lane == 0) {
        const uint64_t t0 = globaltimer();
        do {
          there = ld_acquire(arrived) == 4u * (unsigned)p.nt;
        } while (!there && globaltimer() - t0 < JOIN_WAIT_NS);
      }
      there = __shfl_sync(0xffffffffu, there, 0);
      // `units` of rows to be taken, a ticket each.  A warp's last ticket is one that finds nothing left; those that gave up
      // count in the upper half.  Whoever sees all warps of the sharers in one of the two clears the words for the next launch.
      auto last_of = [&](unsigned before, int units) {
        const int fails = max((int)(before & 0xffffu) - units, 0), gave_up = (int)(before >> 16);
        if (fails + gave_up + 1 == 4 * count) {
          *tickets = 0u;
          *arrived = 0u;
        }
      };
      // ROWS rows at a time, PIECES pieces of each: eight loads under way.  The next ticket is asked for beside them.
      auto join = [&](auto rows_, auto pieces_) {
        constexpr int ROWS = decltype(rows_)::value, PIECES = decltype(pieces_)::value;
        const int units = (R + ROWS - 1) / ROWS;
        unsigned v = 0;
        if (lane == 0) v = atomicAdd(tickets, 1u);
        for (;;) {
          const int unit = (int)(__shfl_sync(0xffffffffu, v, 0) & 0xffffu);
          if (unit >= units) break;
          if (lane == 0) v = atomicAdd(tickets, 1u);
          const int r0 = unit * ROWS;
          float top[ROWS], sum[ROWS];
          float4 acc[ROWS];
#pragma unroll
          for (int i = 0; i < ROWS; ++i) {
            top[i] = -INFINITY;
            sum[i] = 0.f;
            acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
          }
          Sharers s = all;
          for (int base = c_first;; base += 32) {
            while (s.has) {
              float4 u[PIECES][ROWS];
              float2 ml[PIECES][ROWS];
#pragma unroll
              for (int j = 0; j < PIECES; ++j) {
                const int c = s.has ? base + __ffs(s.has) - 1 : -1;
                s.has &= s.has - 1;
#pragma unroll
                for (int i = 0; i < ROWS; ++i) {
                  ml[j][i] = make_float2(-INFINITY, 0.f);
                  u[j][i] = make_float4(0.f, 0.f, 0.f, 0.f);
                  if (c >= 0 && r0 + i < R) {
                    const size_t at = ((size_t)c * 2 + (c == c_first ? 1 : 0)) * MAXR + r0 + i;
                    ml[j][i] = __ldcg(a.part_ml + at);
                    u[j][i] = __ldcg(reinterpret_cast<const float4*>(a.part_o + at * D) + lane);
                  }
                }
              }
#pragma unroll
              for (int i = 0; i < ROWS; ++i) {
                float high = top[i];
#pragma unroll
                for (int j = 0; j < PIECES; ++j) high = fmaxf(high, ml[j][i].x);
                const float base_m = high == -INFINITY ? 0.f : high, keep = ex2(top[i] - base_m);
                sum[i] *= keep;
                acc[i].x *= keep;
                acc[i].y *= keep;
                acc[i].z *= keep;
                acc[i].w *= keep;
                top[i] = high;
#pragma unroll
                for (int j = 0; j < PIECES; ++j) {
                  const float w = ex2(ml[j][i].x - base_m);
                  sum[i] += ml[j][i].y * w;
                  acc[i].x += u[j][i].x * w;
                  acc[i].y += u[j][i].y * w;
                  acc[i].z += u[j][i].z * w;
                  acc[i].w += u[j][i].w * w;
                }
              }
            }
            if (s.t >= p.nt) break;
            s = sharers(base + 32, s.t);
          }
#pragma unroll
          for (int i = 0; i < ROWS; ++i) {
            if (r0 + i >= R) break;
            const float inv = Q4_TILE_SCALE / sum[i];
            const int tok = s_tok[r0 + i], g = r0 + i - tok * a.G;
            *reinterpret_cast<uint2*>(a.O + (size_t)(p.row0 + tok) * a.ldo + (size_t)(p.h * a.G + g) * D + lane * 4) =
                make_uint2(pack_bf16x2(acc[i].x * inv, acc[i].y * inv), pack_bf16x2(acc[i].z * inv, acc[i].w * inv));
          }
        }
        if (lane == 0) last_of(v, units);
      };
      // A quarter of a row's dims at a time, its pieces dealt to four groups of eight lanes, which are joined at the end: 32
      // pieces under way.  For many pieces of few rows (each piece brings four warps): one sequence of one kv head, 8 query
      // heads, at 100000 keys 19.2 us, by whole rows 24.0; of 8 kv heads, 4 rows each, at 8000 keys 11.7 and 13.6.
      auto join_quarters = [&]() {
        const int units = 4 * R, sub = lane >> 3;
        unsigned v = 0;
        if (lane == 0) v = atomicAdd(tickets, 1u);
        for (;;) {
          const int unit = (int)(__shfl_sync(0xffffffffu, v, 0) & 0xffffu);
          if (unit >= units) break;
          if (lane == 0) v = atomicAdd(tickets, 1u);
          const int r = unit >> 2, d = (unit & 3) * 32 + (lane & 7) * 4;
          float top = -INFINITY, sum = 0.f;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
          auto add_piece = [&](float4 u, float2 ml, float base_m) {
            const float w = ex2(ml.x - base_m);
            sum += ml.y * w;
            acc.x += u.x * w;
            acc.y += u.y * w;
            acc.z += u.z * w;
            acc.w += u.w * w;
          };
          auto lift = [&](float high) {
            const float base_m = high == -INFINITY ? 0.f : high, keep = ex2(top - base_m);
            sum *= keep;
            acc.x *= keep;
            acc.y *= keep;
            acc.z *= keep;
            acc.w *= keep;
            top = high;
            return base_m;
          };
          Sharers s = all;
          for (int base = c_first;; base += 32) {
            const int rank = __popc(s.has & ((1u << lane) - 1u));
            unsigned mine = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const unsigned of_k = __ballot_sync(0xffffffffu, (s.has >> lane & 1u) && (rank & 3) == k);
              if (sub == k) mine = of_k;
            }
            float4 u[8];
            float2 ml[8];
            float high = top;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              ml[j] = make_float2(-INFINITY, 0.f);
              u[j] = make_float4(0.f, 0.f, 0.f, 0.f);
              if (mine) {
                const int c = base + __ffs(mine) - 1;
                const size_t at = ((size_t)c * 2 + (c == c_first ? 1 : 0)) * MAXR + r;
                ml[j] = __ldcg(a.part_ml + at);
                u[j] = __ldcg(reinterpret_cast<const float4*>(a.part_o + at * D + d));
              }
              mine &= mine - 1;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) high = fmaxf(high, ml[j].x);
            const float base_m = lift(high);
#pragma unroll
            for (int j = 0; j < 8; ++j) add_piece(u[j], ml[j], base_m);
            if (s.t >= p.nt) break;
            s = sharers(base + 32, s.t);
          }
#pragma unroll
          for (int o = 8; o < 32; o <<= 1) {
            float2 ml;
            float4 u;
            ml.x = __shfl_xor_sync(0xffffffffu, top, o);
            ml.y = __shfl_xor_sync(0xffffffffu, sum, o);
            u.x = __shfl_xor_sync(0xffffffffu, acc.x, o);
            u.y = __shfl_xor_sync(0xffffffffu, acc.y, o);
            u.z = __shfl_xor_sync(0xffffffffu, acc.z, o);
            u.w = __shfl_xor_sync(0xffffffffu, acc.w, o);
            add_piece(u, ml, lift(fmaxf(top, ml.x)));
          }
          if (sub == 0) {
            const float inv = Q4_TILE_SCALE / sum;
            const int tok = s_tok[r], g = r - tok * a.G;
            *reinterpret_cast<uint2*>(a.O + (size_t)(p.row0 + tok) * a.ldo + (size_t)(p.h * a.G + g) * D + d) =
                make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
          }
        }
        if (lane == 0) last_of(v, units);
      };
      const bool quarters = count > 8 && count >= R;
      if (there) {
        __syncwarp();
        if (count == 2) join(Int<4>{}, Int<2>{});
        else if (quarters) join_quarters();
        else join(Int<1>{}, Int<8>{});
      } else if (lane == 0) {
        last_of(atomicAdd(tickets, 0x10000u), count == 2 ? (R + 3) / 4 : quarters ? 4 * R : R);
      }
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(0, TMEM_COLS);
  }
}

template <int NC>
cudaError_t launch(const CUtensorMap& tq, const ChunkAttnArgs& a, int grid, cudaStream_t s) {
  static bool configured[64] = {};
  constexpr int SMEM = Layout<NC>::SMEM;
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !configured[dev]) {
    cudaError_t e = cudaFuncSetAttribute(few_attention_q4_kernel<NC>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != cudaSuccess) return e;
    // the split of registers between the warpgroups draws on what the launch has
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, few_attention_q4_kernel<NC>);
    if (e != cudaSuccess) return e;
    if (fa.numRegs < REGS_ALL) return cudaErrorLaunchOutOfResources;
    if (dev >= 0 && dev < 64) configured[dev] = true;
  }
  cudaError_t e = launch_k(few_attention_q4_kernel<NC>, dim3(grid), dim3(THREADS), SMEM, s, tq, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

// Up to 64 rows (TMEM has 64 columns for a slot's scores) this kernel is the faster one, with few exceptions (in us, this one /
// attention_chunk.cu's; 32 query and 8 kv heads): 64 sequences of 4000 keys with 16 rows per kv head 67 / 144, with 32 80 /
// 144, with 48 93 / 145, with 64 119 / 145; 8 of 30000 keys 60 / 129, 71 / 130, 82 / 130, 108 / 129.  The exceptions: batches
// that give the other's CTAs about one short item each, 8 to 16 sequences of 500 to 1000 keys, with 48 rows up to 4 us, with
// 64 up to 8 (16 at 1000 keys 25.9 / 18.5); the host does not know the lengths.
int few_attention_q4_columns(int G, int max_rows) {
  return (long long)G * max_rows <= MAXR ? (G * max_rows + 15) / 16 * 16 : 0;
}
float q4_tile_scale() { return Q4_TILE_SCALE; }

cudaError_t launch_few_attention_q4(const CUtensorMap& tq, const ChunkAttnArgs& a, int columns, int grid, cudaStream_t s) {
  switch (columns) {
    case 16: return launch<16>(tq, a, grid, s);
    case 32: return launch<32>(tq, a, grid, s);
    case 48: return launch<48>(tq, a, grid, s);
    default: return launch<64>(tq, a, grid, s);
  }
}

}  // namespace spec
