// Attention of a chunk of new tokens over the paged cache on tcgen05 tensor cores: row j of sequence b
// attends keys 0 .. ctx_b + j of its pages (the chunk's own keys are already in them).
//
// Rows.  The G query heads of a kv head share its keys, so a row tile packs TPT = 128 / G tokens x G
// heads (row m = token m / G, head m % G) into the MMA's 128 rows; an item is two row tiles (2 TPT
// tokens of one sequence and kv head) over all key tiles (one page, 128 keys) that its last token sees.
//   S[row, key] = Q . K_tile^T    tcgen05.mma M = 128, N = 128 keys, K = 128 dims (smem x smem)
//   softmax                       one thread per row: running reference and sum in registers, fp32
//   O[row, d]  += P . V_tile      tcgen05.mma M = 128, N = 128 dims, K = 128 keys, P (bf16) read
//                                 from TMEM, where it replaces the scores it came from
// TMEM holds S and O of two slots (4 x 128 columns, all of it).  The steps of a CTA alternate between the
// slots, so that one slot's softmax runs beside the other slot's products.  An item of two row tiles
// gives each slot one of them and both use every key tile (one load, two products); an item with a single
// row tile (few rows: decode steps, ends of prompts) gives the slots its key tiles in turn, each
// with its own reference, sum and O, joined at the end.
//
// Work.  Where the items come out about even (prompts), whole items, the longest first, are dealt to the CTAs in rows
// that run forth and back.  Otherwise the key tiles of all items in a row (sequence, kv head, item) are cut into
// equal shares by cost, one per CTA; without that a prompt's chunk over a long cache would leave a
// wave half empty, and a few rows all but a few CTAs idle.  Where a cut falls into an item its pieces go to the
// workspace as unnormalised O, reference and sum; the warps of the item's CTAs that are done when the last
// piece arrives join it together, in CTA order whoever does it (a second kernel for this took 5 to 8 us
// longer).  Every CTA works all of this out from the lengths on the device (closed form per
// sequence), so one graph serves any lengths.
//
// Bound.  With many rows, the tensor cores: a key tile's four products of 128^3 take 2048 of their cycles, in which
// the softmax warps have to form 256 x 128 weights, which is why nothing else is in their way: a
// maximum once per row (the reference below), two fp32 operations per instruction, a row per thread.  A prompt of 8192 rows
// (32 + 2 x 8 heads) takes 317 us = 1735 TFLOP/s, 2048 rows at 30000 keys 655 us = 1590.  With few rows, HBM: 61 rows
// at 131000 keys 97 to 101 us = 5.4 TB/s, 16 x 32 rows at 4000 keys 47 us = 5.8 TB/s.  (That is for some tens of calls. In
// seconds of them the power limit takes the clock from 2.05 to 1.7 GHz and below: 330 to 360 us for the prompt,
// 106 to 112 us for the 61 rows, from a graph and called one by one alike.)  In between and below, what a
// call costs whatever its size: 4 to 5 us to the first product (lengths, the CTA's pieces, page table, first
// tiles) and, where items are shared, about 8 us to join them; one token of 4 sequences (13.0 us) pays the first,
// a chunk of 512 at 7680 keys (55 us) both.
//
// Roles (12 warps): 0-3 and 4-7 softmax and epilogue of slot 0 and 1 (thread = TMEM lane = row); 8 loads K
// and V tiles by TMA into one ring of 5; 9 issues the MMAs; 10 loads the Q tiles and zeroes the rows of
// a sequence's last V tile behind its last key (up to the next multiple of 16, where the product
// stops), which may hold anything (0 * NaN would reach the sums); 11 walks the batch and posts each of
// the CTA's pieces (consecutive key tiles of one item) to a small ring that the others read, so that
// none of them waits for the lengths or keeps a walk in registers.
#include "common.cuh"
#include "internal.h"

#include <climits>

namespace spec {
namespace {

constexpr int D = 128;
constexpr int KT = 128;                   // keys per tile (one page)
constexpr int TM = 128;                   // rows per row tile
constexpr int ST = 5;                     // ring stages of one K or V tile
constexpr int HALF = 128 * 128;           // 128 rows x 64 bf16 (128-byte swizzled rows), 16 KB
constexpr int TILE = 2 * HALF;
constexpr int THREADS = 384;
constexpr int REGS_ALL = 168, REGS_SOFTMAX = 208, REGS_OTHER = 80;
static_assert(256 * REGS_SOFTMAX + 128 * REGS_OTHER <= THREADS * REGS_ALL, "register split");
constexpr int OFF_Q = 0;                  // two row tiles
constexpr int OFF_RING = 2 * TILE;
constexpr int OFF_BAR = OFF_RING + ST * TILE;
constexpr int PR = 4;                     // posted pieces
constexpr int N_BARS = 3 * ST + 18 + 2 * PR;
constexpr int OFF_RINGP = OFF_BAR + (N_BARS + 1) * 8;   // posted pieces
constexpr int OFF_ML = OFF_BAR + 1024;    // (max, sum) of 128 rows for each slot
constexpr int SMEM = OFF_ML + 2 * TM * 8;
static_assert(SMEM <= 227 * 1024, "shared memory budget");
constexpr uint32_t TMEM_COLS = 512;       // S0 S1 O0 O1

constexpr uint64_t JOIN_WAIT_NS = 20000;  // how long a warp that is done waits for the other pieces of a shared item
// Cost of a key for an item of two row tiles and of one, and what an item's start and end cost in keys; the time that
// joining shared items takes at the end, in keys of two row tiles; what reading a piece back takes, in keys of one.
constexpr int W_DUAL = 4, W_ONE = 3, ITEM_KEYS = 384, JOIN_KEYS = 1280, PIECE_KEYS = 36;

// 128 consecutive TMEM columns of this thread's lane, loaded and waited for in one asm
__device__ __forceinline__ void tmem_ld_cols128(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%128+0];\n"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%128+32];\n"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%64,%65,%66,%67,%68,%69,%70,%71,%72,%73,%74,%75,%76,%77,%78,%79,%80,%81,%82,%83,%84,%85,%86,%87,%88,%89,%90,%91,%92,%93,%94,%95}, [%128+64];\n"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%96,%97,%98,%99,%100,%101,%102,%103,%104,%105,%106,%107,%108,%109,%110,%111,%112,%113,%114,%115,%116,%117,%118,%119,%120,%121,%122,%123,%124,%125,%126,%127}, [%128+96];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63]), "=r"(r[64]), "=r"(r[65]), "=r"(r[66]), "=r"(r[67]), "=r"(r[68]), "=r"(r[69]), "=r"(r[70]), "=r"(r[71]), "=r"(r[72]), "=r"(r[73]), "=r"(r[74]), "=r"(r[75]), "=r"(r[76]), "=r"(r[77]), "=r"(r[78]), "=r"(r[79]), "=r"(r[80]), "=r"(r[81]), "=r"(r[82]), "=r"(r[83]), "=r"(r[84]), "=r"(r[85]), "=r"(r[86]), "=r"(r[87]), "=r"(r[88]), "=r"(r[89]), "=r"(r[90]), "=r"(r[91]), "=r"(r[92]), "=r"(r[93]), "=r"(r[94]), "=r"(r[95]), "=r"(r[96]), "=r"(r[97]), "=r"(r[98]), "=r"(r[99]), "=r"(r[100]), "=r"(r[101]), "=r"(r[102]), "=r"(r[103]), "=r"(r[104]), "=r"(r[105]), "=r"(r[106]), "=r"(r[107]), "=r"(r[108]), "=r"(r[109]), "=r"(r[110]), "=r"(r[111]), "=r"(r[112]), "=r"(r[113]), "=r"(r[114]), "=r"(r[115]), "=r"(r[116]), "=r"(r[117]), "=r"(r[118]), "=r"(r[119]), "=r"(r[120]), "=r"(r[121]), "=r"(r[122]), "=r"(r[123]), "=r"(r[124]), "=r"(r[125]), "=r"(r[126]), "=r"(r[127])
      : "r"(taddr)
      : "memory");
}

// 32 consecutive TMEM columns of this thread's lane stored (complete after tmem_st_wait)
__device__ __forceinline__ void tmem_st_cols32(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
               : "memory");
}
__device__ __forceinline__ void tmem_st_cols16(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
                   taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
               "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D += A B with A (bf16, two consecutive k per 32-bit column) in TMEM.
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// ... only if `go` (a predicated instruction, not a branch).
__device__ __forceinline__ void umma_bf16_ts_if(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                                bool go) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 q, %4, 0;\n setp.eq.u32 p, 0, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"((uint32_t)go)
      : "memory");
}
// Shared-memory descriptor of an MN-major operand stored as 128-byte swizzled rows (8-row atoms 1024 B
// apart along K; 64-element columns `lbo` apart along N).
__device__ __forceinline__ uint64_t desc_mn(uint32_t smem_addr, uint32_t lbo) {
  uint64_t d = 0;
  d |= uint64_t((smem_addr & 0x3FFFFu) >> 4);
  d |= uint64_t((lbo >> 4) & 0x3FFFu) << 16;
  d |= uint64_t(1024 >> 4) << 32;
  d |= uint64_t(1) << 46;
  d |= uint64_t(2) << 61;
  return d;
}
__device__ __forceinline__ unsigned ld_acquire(const unsigned* p) {
  unsigned v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void red_release(unsigned* p, unsigned v) {
  asm volatile("red.release.gpu.global.add.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
// 2^x on the special-function unit (relative error about 2^-22; 2^-inf = 0)
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t cvt_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// The library's bounded wait, short: thirty of them are in this kernel, and what runs once per piece runs from a
// cold instruction cache.  Each role tells the status word itself when one ran out.
// (The limit is in cycles, a second or more at the chip's clocks: the wall clock takes long to read.)
constexpr uint32_t WAIT_CYCLES = 1u << 31;
__device__ __forceinline__ uint32_t cycles() {
  uint32_t t;
  asm volatile("mov.u32 %0, %clock;" : "=r"(t));
  return t;
}
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint32_t t0 = cycles();
  do {
    if (mbar_try_wait(bar, parity)) return true;
  } while (cycles() - t0 < WAIT_CYCLES);
  return false;
}
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
      " fma.rn.f32x2 x, x, y, z;\n mov.b64 {%0, %1}, x;\n}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n .reg .b64 x, y;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n"
      " add.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

// 32 bytes to a 32-byte boundary: a row per lane then fills whole sectors (as 16-byte stores the outputs of a prompt of
// 8192 rows took 24 us more; exchanged between lanes first to fill lines, 8 us more).  Past L1, whose lines the 32 rows
// of a warp would take one each (8 prompts of 500 rows 30.9 us without the hint, 28.1 with it).
__device__ __forceinline__ void st_global_32(void* p, const uint32_t* w) {
  asm volatile("st.global.L1::no_allocate.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]),
               "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ void st_global_16(void* p, const uint32_t* w) {      // (outputs at odd 16 bytes)
  asm volatile("st.global.L1::no_allocate.v4.b32 [%0], {%1,%2,%3,%4};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3])
               : "memory");
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
  const bool ok = c0 >= 0 && c1 >= c0 && c1 <= a.M &&
                  (c0 == c1 || (ctx >= 0 && (long long)ctx + (c1 - c0) <= (long long)a.max_pages * KT));
  if (bad) *bad = !ok;
  return Seq{c0, ok ? c1 - c0 : 0, ctx};
}
// n / T for n <= 2^22 (T = 2 tpt <= 256; t_magic = floor(2^32 / T) + 1)
__device__ __forceinline__ int div_t(const ChunkAttnArgs& a, int n) { return (int)__umulhi((unsigned)n, a.t_magic); }
// Cost of the first q items (all of two row tiles) of one kv head of a sequence: item i sees
// ctx + (i + 1) T keys.
__device__ __forceinline__ long long items_cost(int q, int T, int ctx) {
  return W_DUAL * ((long long)q * (ctx + ITEM_KEYS) + (long long)q * (q + 1) / 2 * T);
}
// ... and of all its items.
__device__ __forceinline__ long long head_cost(const ChunkAttnArgs& a, const Seq& s) {
  if (s.rows == 0) return 0;
  const int T = 2 * a.tpt, last = div_t(a, s.rows - 1);
  const int w = s.rows - last * T > a.tpt ? W_DUAL : W_ONE;
  return items_cost(last, T, s.ctx) + (long long)w * (s.ctx + s.rows + ITEM_KEYS);
}
// The tile that a cut at cost y of an item (its start 0) falls before: 0 .. nt.
__device__ __forceinline__ int cut_tile(long long y, bool dual, int keys, int nt) {
  const int w = dual ? W_DUAL : W_ONE;
  y -= w * ITEM_KEYS;
  if (y <= 0) return 0;
  if (y >= (long long)w * keys) return nt;
  const unsigned z = dual ? (unsigned)y / W_DUAL : (unsigned)y / W_ONE;      // (keys <= 2^30)
  const int t = (int)((z + KT / 2) / KT);
  return t * KT + KT / 2 >= keys ? nt : t;              // (no piece of a few keys)
}
// The cost of the batch and of a CTA's share of it (the last ones' may be smaller or nothing).
struct Shares {
  long long total, each;
  __device__ __forceinline__ long long start(int c) const { return min(total, c * each); }
};
// Equal shares, but of so many keys that an item's pieces are not joined for longer than they take: with `keys` of the
// longest item and a piece's reading back as long as PIECE_KEYS, n sharers take keys / n and n PIECE_KEYS (9 rows of 5
// heads at 63118 keys: 63 us with 152 sharers, 27.6 with 42).  inv_grid = floor((2^64 - 1) / grid).
__device__ __forceinline__ Shares shares_of(const ChunkAttnArgs& a, long long total, int keys) {
  const long long even = (long long)__umul64hi((unsigned long long)total, a.inv_grid) + 1;
  return Shares{total, max(even, (long long)(W_ONE * sqrtf((float)PIECE_KEYS * keys)))};
}

// Where a cut falls: before tile t of item q of kv head h of sequence b (which is s); `start`: the cost of
// everything before the item.
struct Cut {
  long long start;
  int b, h, q, t;
  Seq s;
};
// A cut at cost x of sequence b (0 <= x < cost of all its heads; `before`: of everything before it).
struct Found {
  long long x, before;
  int b;
  Seq s;
};
// The cut on a whole tile, by 16 lanes.
__device__ __forceinline__ Cut cut_of(const ChunkAttnArgs& a, const Found& f, int lane) {
  const int T = 2 * a.tpt;
  Cut c;
  c.b = f.b;
  c.s = f.s;
  c.h = c.q = c.t = 0;
  long long x = f.x;
  int lo = 0, n = 0;
  if (f.s.rows > 0) {
    const long long head = head_cost(a, f.s);
    int h = (int)__fdividef(__ll2float_rz(x), __ll2float_ru(head));      // (off by one at most, then put right)
    h = h < a.Hkv ? h : a.Hkv - 1;
    while (h > 0 && h * head > x) --h;
    while ((h + 1) * head <= x) ++h;
    c.h = h;
    x -= h * head;
    n = div_t(a, f.s.rows - 1) + 1;
  }
  // the last item that starts at or before x: 16 candidates at a time
  while (__any_sync(0xffffffffu, n > 1)) {
    const int step = (n + 15) >> 4, q = lo + (lane & 15) * step;
    const unsigned votes = __ballot_sync(0xffffffffu, n > 1 && q < lo + n && items_cost(q, T, f.s.ctx) <= x);
    if (n > 1) {
      const int k = 31 - __clz((votes >> (lane & 16)) & 0xffffu);      // (the first always is)
      n = min(step, n - k * step);
      lo += k * step;
    }
  }
  if (f.s.rows > 0) {
    c.q = lo;
    x -= items_cost(lo, T, f.s.ctx);
    const int tok = min(T, f.s.rows - lo * T), keys = f.s.ctx + lo * T + tok;
    c.t = cut_tile(x, tok > a.tpt, keys, (keys + KT - 1) / KT);
  }
  c.start = f.before + f.x - x;
  return c;
}

// Items of one kv head of a sequence that see x keys or more (x >= 1; keys = ctx + rows, 0 without rows).
__device__ __forceinline__ int items_from(const ChunkAttnArgs& a, int rows, int keys, int x) {
  if (x > keys) return 0;
  const int last = div_t(a, rows - 1);
  return last + 1 - min(div_t(a, max(x - 1 - (keys - rows), 0)), last);
}

// A CTA's consecutive key tiles of one item, as posted.
struct Piece {
  int b, h, q;
  int t0, t1, nt;      // tiles t0 .. t1 - 1 of the item's nt
  int row0;            // first packed row
  int tok, pos;        // tokens of the item, position of the first
  int dual;            // two row tiles
  int once;            // the sequence's only item of this head: its keys are read once
  int more;            // 0: no piece, the CTA is done
  long long start;     // cost of everything before the item (where a cut falls into it)

  __device__ __forceinline__ int tiles() const { return t1 - t0; }
  // the piece in pairs of steps (slot 0, slot 1); the second of the last pair may be void
  __device__ __forceinline__ int pairs() const { return dual ? tiles() : (tiles() + 1) >> 1; }
  // steps of a slot, and the key tile of its j-th
  __device__ __forceinline__ int steps(int sl) const { return dual ? tiles() : (tiles() + 1 - sl) >> 1; }
  __device__ __forceinline__ int tile(int sl, int j) const { return t0 + (dual ? j : 2 * j + sl); }
  __device__ __forceinline__ int keys() const { return pos + tok; }
  __device__ __forceinline__ bool tail() const { return t1 == nt && (keys() & 15) != 0; }
};
static_assert(OFF_RINGP + (PR + 1) * sizeof(Piece) + sizeof(Shares) <= OFF_ML && OFF_RINGP % 8 == 0, "posted pieces");

// The walk over a CTA's pieces, by a whole warp.
struct Walk {
  Piece p;
  Seq s;
  __device__ __forceinline__ void item(int T) {
    p.start = 0;
    p.tok = min(T, s.rows - p.q * T);
    p.row0 = s.r0 + p.q * T;
    p.pos = s.ctx + p.q * T;
    p.nt = (p.pos + p.tok + KT - 1) / KT;
    p.dual = p.tok > T / 2;
    p.once = s.rows <= T;
  }
  // the piece ends at the item's end or at the CTA's
  __device__ __forceinline__ void clip(const Cut& e) {
    p.t1 = p.nt;
    if (p.b == e.b && p.h == e.h && p.q == e.q) {
      p.t1 = e.t;
      p.start = e.start;
    } else if (p.b > e.b || (p.b == e.b && (p.h > e.h || (p.h == e.h && p.q > e.q)))) p.t1 = 0;
    p.more = p.t1 > p.t0;
  }
  // first piece of [c, e)
  __device__ __forceinline__ void first(const ChunkAttnArgs& a, const Cut& c, const Cut& e, int lane) {
    p.more = 0;
    if (c.b >= a.B) return;
    p.b = c.b; p.h = c.h; p.q = c.q; p.t0 = c.t;
    s = c.s;
    item(2 * a.tpt);
    p.start = c.start;
    if (p.t0 >= p.nt) next(a, e, lane);
    else clip(e);
  }
  __device__ __forceinline__ void next(const ChunkAttnArgs& a, const Cut& e, int lane) {
    p.t0 = 0;
    p.more = 0;
    if (++p.q * 2 * a.tpt >= s.rows) {
      p.q = 0;
      if (++p.h == a.Hkv) {
        p.h = 0;
        // the next sequence with rows, 32 candidates at a time (a padded batch may have hundreds without)
        for (int from = p.b + 1;; from += 32) {
          if (from >= a.B || from > e.b) return;
          const Seq c = from + lane < a.B ? seq_of(a, from + lane) : Seq{0, 0, 0};
          const unsigned has = __ballot_sync(0xffffffffu, c.rows > 0);
          if (has == 0) continue;
          const int k = __ffs(has) - 1;
          p.b = from + k;
          s.r0 = __shfl_sync(0xffffffffu, c.r0, k);
          s.rows = __shfl_sync(0xffffffffu, c.rows, k);
          s.ctx = __shfl_sync(0xffffffffu, c.ctx, k);
          break;
        }
      }
    }
    item(2 * a.tpt);
    clip(e);
  }
};

__global__ void __launch_bounds__(THREADS, 1)
chunk_attention_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const ChunkAttnArgs a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
  uint64_t* full = bars;                   // [ST] tile ready
  uint64_t* empty = full + ST;             // [ST] its products done
  uint64_t* land = empty + ST;             // [ST] load landed of a V tile whose end is to be zeroed
  uint64_t* q_full = land + ST;            // [2]  row tile of a slot ready
  uint64_t* q_empty = q_full + 2;          // [2]  its last Q K^T of a piece done
  uint64_t* s_full = q_empty + 2;          // [2]  scores in TMEM (and the slot's P V before them done)
  uint64_t* p_full = s_full + 2;           // [2]  P in TMEM, O rescaled
  uint64_t* o_full = p_full + 2;           // [2]  last P V of a piece done
  uint64_t* pair = o_full + 2;             // [4][2] the warps of both slots with the same rows: sums exchanged, O read
  uint64_t* posted = pair + 8;             // [PR] piece posted
  uint64_t* taken = posted + PR;           // [PR] everyone is done with its entry
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + N_BARS);
  Piece* ring = reinterpret_cast<Piece*>(smem + OFF_RINGP);
  Piece* s_first = ring + PR;              // the CTA's first piece, for the end
  Shares* s_shares = reinterpret_cast<Shares*>(ring + PR + 1);
  float2* s_ml = reinterpret_cast<float2*>(smem + OFF_ML);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if ((smem_u32(smem) & 1023u) != 0) {     // (the swizzled tiles need it; the same for every thread)
    if (tid == 0) set_status(a.status, 0x7F3u);
    return;
  }
  if (tid == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    for (int i = 0; i < 3 * ST; ++i) mbar_init(&bars[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&o_full[i], 1);
    }
    for (int i = 0; i < 8; ++i) mbar_init(&pair[i], 2);
    for (int i = 0; i < PR; ++i) {
      mbar_init(&posted[i], 1);
      mbar_init(&taken[i], 11);              // loads, MMA, Q tiles, 8 softmax warps
    }
    fence_barrier_init();
  }
  if (warp == 9) tmem_alloc(tmem_slot, TMEM_COLS);

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  constexpr uint32_t tmem = 0;             // (all 512 columns are this CTA's)
  if (*tmem_slot != tmem && tid == 0) set_status(a.status, 0x7F4u);
  // everything above overlaps the kernel before; global memory only below
  pdl_wait();
  pdl_trigger();

  // the softmax warps hold a row of scores each: the other warpgroup leaves them its registers
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_OTHER));
    if (warp == 11) {
      // ------------------------------------------------------------ pieces
      // The sequences, a run of them per lane.
      const int run = (a.B + 31) >> 5, b0 = min(lane * run, a.B), b1 = min(b0 + run, a.B);
      long long own = 0;
      bool bad = false;
      Seq mine{0, 0, 0};
      int longest = 0;
#pragma unroll 4
      for (int b = b0; b < b1; ++b) {
        bool wrong;
        mine = seq_of(a, b, &wrong);
        bad |= wrong;
        own += head_cost(a, mine) * a.Hkv;
        if (mine.rows > 0) longest = max(longest, mine.ctx + mine.rows);
      }
      if (bad && blockIdx.x == 0) set_status(a.status, 0x7F1u);
      // Where they come out about even, whole items, the longest first, dealt to the CTAs in rows that run forth and
      // back: nothing is left to join.  (8 prompts of 100 to 1900 rows 40.4 us, cut 53.5; one of 2048 rows 29.2,
      // cut 42.6; of 8192 rows 317, cut 335; 16 x 32 rows at 4000 keys 46.8, cut 53.9.)  What the deal leaves uneven
      // is about the longest item of the last row times the share of the CTAs that the row leaves out: the rule is
      // that this costs less than joining.  Over 20 batches it took the faster side, or one within 1 us of it.  Items of
      // one tile are never cut.
      const int T = 2 * a.tpt, grid = (int)gridDim.x;
      const int keys = longest;              // (of the lane's one sequence, below)
      const int items = run > 1 ? 0 : __reduce_add_sync(0xffffffffu, items_from(a, mine.rows, keys, 1)) * a.Hkv;
      bool whole = false;
      if (__any_sync(0xffffffffu, longest > KT) && items > 0) {
        const int before = (items - 1) / grid * grid, out = grid - (items - before);
        const int x = out == 0 ? INT_MAX : JOIN_KEYS * grid / out - ITEM_KEYS + 1;
        whole = __reduce_add_sync(0xffffffffu, items_from(a, mine.rows, keys, x)) * a.Hkv <= before;
      }
      // the k-th piece to the others; false after a wait that ran out
      auto post = [&](int k, const Piece& p) {
        const bool ok = k < PR || wait_for(&taken[k % PR], (uint32_t)((k / PR - 1) & 1));
        if (!__all_sync(0xffffffffu, ok)) {
          if (lane == 0) set_status(a.status, 0x701u);
          return false;
        }
        if (lane == 0) {
          ring[k % PR] = p;
          mbar_arrive(&posted[k % PR]);
        }
        __syncwarp();
        return true;
      };
      if (whole) {
        Walk w;
        int x = 1, n = (int)__reduce_max_sync(0xffffffffu, (unsigned)keys);
        for (int k = 0;; ++k) {
          const int at = k * grid + ((k & 1) ? grid - 1 - (int)blockIdx.x : (int)blockIdx.x);
          const bool more = at < items;
          if (more) {
            // the most keys that more than `rank` items see, 32 candidates at a time
            const int rank = at / a.Hkv;
            while (n > 1) {
              const int step = (n + 31) >> 5, c = x + lane * step;
              int count = 0;
#pragma unroll 4
              for (int b = 0; b < a.B; ++b)
                count += items_from(a, __shfl_sync(0xffffffffu, mine.rows, b), __shfl_sync(0xffffffffu, keys, b), c);
              const int i = 31 - __clz(__ballot_sync(0xffffffffu, c < x + n && count > rank));   // (the first always)
              n = min(step, n - i * step);
              x += i * step;
            }
            // of the items that see just as many, one per sequence, the one whose turn it is
            const int from = items_from(a, mine.rows, keys, x), above = items_from(a, mine.rows, keys, x + 1);
            const unsigned same = __ballot_sync(0xffffffffu, from > above);
            const int turn = rank - __reduce_add_sync(0xffffffffu, above);
            const bool me = from > above && __popc(same & ((1u << lane) - 1u)) == turn;
            const int b = __ffs(__ballot_sync(0xffffffffu, me)) - 1;
            w.p.b = b;
            w.p.h = at - rank * a.Hkv;
            w.p.q = __shfl_sync(0xffffffffu, items_from(a, mine.rows, keys, 1) - from, b);
            w.s.r0 = __shfl_sync(0xffffffffu, mine.r0, b);
            w.s.rows = __shfl_sync(0xffffffffu, mine.rows, b);
            w.s.ctx = __shfl_sync(0xffffffffu, mine.ctx, b);
            w.item(T);
            n = x;                         // (the next item sees as many at most)
            x = 1;
          }
          w.p.t0 = 0;
          w.p.t1 = w.p.nt;
          w.p.more = more;
          if (!post(k, w.p) || !more) break;
        }
      } else {
        // Equal shares by cost: the two sequences that this CTA's starts and ends in, found by the lanes that have them.
        long long before = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long v = __shfl_up_sync(0xffffffffu, before, o);
          if (lane >= o) before += v;
        }
        const Shares shares = shares_of(a, __shfl_sync(0xffffffffu, before, 31),
                                        (int)__reduce_max_sync(0xffffffffu, (unsigned)longest));
        before -= own;
        Found f{0, 0, a.B, Seq{0, 0, 0}};      // lanes 0-15: of the start, 16-31: of the end
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const long long x = shares.start(blockIdx.x + k);
          const unsigned owner = __ballot_sync(0xffffffffu, x >= before && x < before + own);
          if (owner == 0) continue;            // (the end of everything, or nothing at all)
          Found g{0, before, b0, Seq{0, 0, 0}};
          if (x >= before && x < before + own)
            for (;; ++g.b) {
              g.s = seq_of(a, g.b);
              const long long c = head_cost(a, g.s) * a.Hkv;
              if (x < g.before + c) break;
              g.before += c;
            }
          const int from = __ffs(owner) - 1;
          g.before = __shfl_sync(0xffffffffu, g.before, from);
          g.b = __shfl_sync(0xffffffffu, g.b, from);
          g.s.r0 = __shfl_sync(0xffffffffu, g.s.r0, from);
          g.s.rows = __shfl_sync(0xffffffffu, g.s.rows, from);
          g.s.ctx = __shfl_sync(0xffffffffu, g.s.ctx, from);
          g.x = x - g.before;
          if ((lane >> 4) == k) f = g;
        }
        const Cut cut = cut_of(a, f, lane);
        auto lane_of = [&](int from) {
          Cut c;
          c.start = __shfl_sync(0xffffffffu, cut.start, from);
          c.b = __shfl_sync(0xffffffffu, cut.b, from);
          c.h = __shfl_sync(0xffffffffu, cut.h, from);
          c.q = __shfl_sync(0xffffffffu, cut.q, from);
          c.t = __shfl_sync(0xffffffffu, cut.t, from);
          c.s.r0 = __shfl_sync(0xffffffffu, cut.s.r0, from);
          c.s.rows = __shfl_sync(0xffffffffu, cut.s.rows, from);
          c.s.ctx = __shfl_sync(0xffffffffu, cut.s.ctx, from);
          return c;
        };
        const Cut start = lane_of(0), end = lane_of(16);
        Walk w;
        w.first(a, start, end, lane);
        if (lane == 0) {
          *s_first = w.p;
          *s_shares = shares;
        }
        for (int k = 0; post(k, w.p) && w.p.more; ++k) w.next(a, end, lane);
      }
      __syncwarp();
    } else if (warp == 8) {
      // ------------------------------------------------------------ K and V tiles
      // in the order of their first products: a step's V tile, then the K tile of its slot's next step
      int idx = 0;
      bool ok = true;
      uint32_t landed = 0;                   // stages whose last load signals `land`
      uint32_t n_land = 0;                   // its phase, one bit per stage
      const uint64_t pol = l2_policy_evict_first();
      // page ids of 32 tiles at a time, one per lane
      struct Pages {
        int id, base;
      };
      auto load = [&](const Piece& p, Pages& pg, int t, bool is_v) {
        if (pg.base < 0 || t >= pg.base + 32) {
          pg.base = t;
          pg.id = t + lane < p.t1 ? a.block_table[(size_t)p.b * a.max_pages + t + lane] : 0;
          if (pg.id < 0 || pg.id >= a.num_pages) {
            set_status(a.status, 0x7F2u);
            pg.id = 0;
          }
        }
        const int page = __shfl_sync(0xffffffffu, pg.id, t - pg.base);
        const int st = idx % ST;
        if (idx >= ST) ok = ok && wait_for(&empty[st], (uint32_t)((idx / ST - 1) & 1));
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return;
        const bool tail = is_v && t == p.nt - 1 && p.tail();
        uint64_t* bar = tail ? &land[st] : &full[st];
        if (lane == 0) {
          const CUtensorMap* tm = is_v ? &tmV : &tmK;
          uint8_t* dst = smem + OFF_RING + st * TILE;
          const int z = p.h * a.num_pages + page;
          mbar_arrive_expect_tx(bar, TILE);
          if (p.once) {
            tma_load_3d_hint(dst, tm, bar, 0, 0, z, pol);
            tma_load_3d_hint(dst + HALF, tm, bar, 64, 0, z, pol);
          } else {
            tma_load_3d(dst, tm, bar, 0, 0, z);
            tma_load_3d(dst + HALF, tm, bar, 64, 0, z);
          }
        }
        if (tail) {
          landed |= 1u << st;
          n_land ^= 1u << st;
        } else {
          landed &= ~(1u << st);
        }
        ++idx;
      };
      auto open = [&](int k) {
        ok = ok && wait_for(&posted[k % PR], (uint32_t)((k / PR) & 1));
        ok = __all_sync(0xffffffffu, ok);
        Piece p = ring[k % PR];
        if (!ok) p.more = 0;
        return p;
      };
      // pair by pair (before the first: K only): V and the next K of slot 0, then of slot 1
      Piece p = open(0), nx = p;
      Pages pv{0, -1}, pk{0, -1};
      for (int k = 0, j = -1; ok && nx.more;) {
        const bool ends = j + 1 == p.pairs();
        if (ends) {
          nx = open(k + 1);
          pk.base = -1;
        }
        const int nj = ends ? 0 : j + 1;
#pragma unroll 1
        for (int q = 0; q < 4 && ok; ++q) {
          const int sl = q >> 1;
          const bool is_v = !(q & 1);
          const Piece& from = is_v ? p : nx;
          const int at = is_v ? j : nj;
          if (at >= 0 && from.more && (sl == 0 || !from.dual) && at < from.steps(sl))
            load(from, is_v ? pv : pk, from.tile(sl, at), is_v);
        }
        j = nj;
        if (ends) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&taken[k % PR]);
          ++k;
          p = nx;
          pv.base = -1;
        }
      }
      if (!ok) {                             // gave up: see the copies in flight land before leaving
        set_status(a.status, 0x711u);
        for (int j = idx > ST ? idx - ST : 0; j < idx; ++j) {
          const int st = j % ST;
          if ((landed >> st) & 1u) wait_for(&land[st], ((n_land >> st) & 1u) ^ 1u);
          else wait_for(&full[st], (uint32_t)((j / ST) & 1));
        }
      }
    } else if (warp == 9) {
      // ------------------------------------------------------------ MMA issue
      // The whole warp walks the steps and one elected lane issues: addresses are then the same in every lane
      // (TMEM and Q addresses constants of the slot, the ring stage a uniform count), which the MMAs take
      // from uniform registers.  Issued from a divergent branch each MMA cost 60 to 100 cycles of operand moves,
      // its 64 cycles on the tensor core twice over.  Few MMAs queue, so what the warp does between them
      // leaves the tensor core idle: the tiles of a pair are waited for before its weights, and after a wait that
      // ran out the warp goes on without waiting (to garbage that nobody reads) instead of voting each time.
      const bool leader = elect_one();
      constexpr uint32_t idesc_s = umma_idesc_bf16(TM, KT);
      constexpr uint32_t idesc_pv = umma_idesc_bf16(TM, D) | (1u << 16);   // B (V) MN-major
      const uint64_t q0 = umma_desc_sw128(smem_u32(smem + OFF_Q)), k0 = umma_desc_sw128(smem_u32(smem + OFF_RING));
      const uint64_t v0 = desc_mn(smem_u32(smem + OFF_RING), HALF);
      int st = 0;                            // next ring stage
      uint32_t ph = 0, ph_p = 0, ph_q = 0;   // phases: the ring's; each slot's weights and Q tile, one bit per slot
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (ok) ok = wait_for(bar, parity);
      };
      // the next ring stage and its phase
      struct Stage {
        int st;
        uint32_t ph;
      };
      auto take = [&]() {
        const Stage mine{st, ph};
        if (++st == ST) {
          st = 0;
          ph ^= 1u;
        }
        return mine;
      };
      auto ready = [&](const Stage& t) { return mbar_try_wait(&full[t.st], t.ph); };
      auto wait_tile = [&](const Stage& t) { wait(&full[t.st], t.ph); };
      // scores of a slot from the K tile of stage kst; first / last: of the slot's steps of the piece
      auto scores = [&](const int sl, int kst, bool first, bool last, bool release) {
        if (first) {
          wait(&q_full[sl], (ph_q >> sl) & 1u);
          ph_q ^= 1u << sl;
          tc_fence_after();
        }
        if (leader) {
          const uint64_t qd = q0 + sl * (TILE >> 4), kd = k0 + (uint32_t)(kst * (TILE >> 4));
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {   // (descriptor addresses count 16 bytes)
            const uint32_t off = ((kk >> 2) * HALF + (kk & 3) * 32) >> 4;
            umma_bf16(sl * KT, qd + off, kd + off, idesc_s, kk > 0 ? 1u : 0u);
          }
          umma_commit(&s_full[sl]);
          if (release) umma_commit(&empty[kst]);
          if (last) umma_commit(&q_empty[sl]);
        }
      };
      // O += P V of a slot from the V tile of stage vst, over `steps` times 16 keys
      auto weigh = [&](const int sl, int vst, int steps, bool first, bool last, bool release) {
        if (leader) {
          const uint64_t vd = v0 + (uint32_t)(vst * (TILE >> 4));
          constexpr uint32_t t_o = 2 * KT;
          umma_bf16_ts(t_o + sl * D, sl * KT, vd, idesc_pv, first ? 0u : 1u);
#pragma unroll
          for (int kk = 1; kk < 8; ++kk)
            umma_bf16_ts_if(t_o + sl * D, sl * KT + kk * 8, vd + kk * 128, idesc_pv, kk < steps);
          if (release) umma_commit(&empty[vst]);
          if (last) umma_commit(&o_full[sl]);
        }
      };
      struct Run {                           // what a piece's steps need
        bool more, dual;
        int n0, n1;                          // steps of the slots
        int tail;                            // 16-key steps of its last tile up to the last key
      };
      auto open = [&](int k) {
        wait(&posted[k % PR], (uint32_t)((k / PR) & 1));
        ok = __all_sync(0xffffffffu, ok);
        const Piece& p = ring[k % PR];
        Run r{ok && p.more, p.dual != 0, p.steps(0), p.steps(1), min(8, (p.keys() - (p.t1 - 1) * KT + 15) >> 4)};
        return r;
      };
      // pair by pair (before the first: scores only)
      Run r = open(0), nx = r;
      Stage k_a{0, 0}, k_b{0, 0}, v_a{0, 0}, v_b{0, 0};
      for (int k = 0, j = -1; nx.more;) {
        // two row tiles, and the next pair of the same piece: nothing to decide (with the general case's
        // decisions in the way 2048 rows at 30000 keys took 700 us instead of 650)
        while (r.dual && j >= 0 && j + 1 < r.n0) {
          const Stage v = take(), t = take();
          const uint32_t pa = ph_p & 1u, pb = (ph_p >> 1) & 1u;
          const bool r0 = ready(v), r1 = ready(t), r2 = mbar_try_wait(&p_full[0], pa);
          if (!(r0 && r1 && r2)) {
            wait_tile(v);
            wait_tile(t);
            wait(&p_full[0], pa);
          }
          tc_fence_after();
          weigh(0, v.st, 8, j == 0, false, false);
          scores(0, t.st, false, j + 2 == r.n0, false);
          wait(&p_full[1], pb);
          tc_fence_after();
          weigh(1, v.st, 8, j == 0, false, true);
          scores(1, t.st, false, j + 2 == r.n0, true);
          ph_p ^= 3u;
          ++j;
        }
        const bool ends = j + 1 == r.n0;     // (slot 0 has a step in every pair)
        if (ends) nx = open(k + 1);
        const int nj = ends ? 0 : j + 1;
        const bool now_a = j >= 0, now_b = now_a && j < r.n1, next_a = nx.more, next_b = nx.more && nj < nx.n1;
        const bool last_tile_b = !r.dual && now_b && ends;      // slot 1 holds the piece's last tile
        // one look at all that slot 0 needs; what is not there is waited for in turn
        if (now_a) v_a = take();
        if (next_a) k_a = take();
        const uint32_t pa = ph_p & 1u, pb = (ph_p >> 1) & 1u;
        // (a try that cannot succeed is not made: it holds the warp for microseconds)
        bool all = false;
        if (now_a && next_a) {
          const bool r0 = ready(v_a), r1 = ready(k_a), r2 = mbar_try_wait(&p_full[0], pa);
          all = r0 && r1 && r2;
        }
        if (!all) {
          if (now_a) wait_tile(v_a);
          if (next_a) wait_tile(k_a);
          if (now_a) wait(&p_full[0], pa);
        }
        tc_fence_after();
        if (now_a) {
          weigh(0, v_a.st, ends && !last_tile_b ? r.tail : 8, j == 0, ends, !r.dual);
          ph_p ^= 1u;
        }
        if (next_a) scores(0, k_a.st, nj == 0, nj + 1 == nx.n0, !nx.dual);
        if (now_b) v_b = r.dual ? v_a : take();
        if (next_b) k_b = nx.dual ? k_a : take();
        all = false;
        if (now_b && next_b) {
          const bool s0 = ready(v_b), s1 = ready(k_b), s2 = mbar_try_wait(&p_full[1], pb);
          all = s0 && s1 && s2;
        }
        if (!all) {
          if (now_b) wait_tile(v_b);
          if (next_b) wait_tile(k_b);
          if (now_b) wait(&p_full[1], pb);
        }
        tc_fence_after();
        if (now_b) {
          weigh(1, v_b.st, ends ? r.tail : 8, j == 0, j + 1 == r.n1, true);
          ph_p ^= 2u;
        }
        if (next_b) scores(1, k_b.st, nj == 0, nj + 1 == nx.n1, true);
        j = nj;
        if (ends) {
          __syncwarp();
          if (leader) mbar_arrive(&taken[k % PR]);
          ++k;
          r = nx;
        }
      }
      if (!ok) set_status(a.status, 0x721u);
      __syncwarp();
    } else {
      // ------------------------------------------------------------ Q tiles, ends of the last V tiles
      uint32_t n_q[2] = {0, 0}, n_land = 0;
      int tiles = 0;                         // key tiles of the pieces so far
      const uint32_t q_bytes = (uint32_t)(a.tpt * a.G * D * 2);
      bool ok = true, had = false, more = true;
      for (int k = 0; (more || had) && ok; ++k) {
        const Piece* p = ring + k % PR;
        const Piece* before = ring + (k + PR - 1) % PR;
        if (more) {
          ok = __all_sync(0xffffffffu, wait_for(&posted[k % PR], (uint32_t)((k / PR) & 1)));
          if (!ok) break;
          more = p->more != 0;
        }
        if (more) {
          for (int sl = 0; sl < 2 && p->steps(sl) > 0; ++sl) {
            if (n_q[sl] > 0) ok = ok && wait_for(&q_empty[sl], (n_q[sl] - 1) & 1);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            ++n_q[sl];
            if (lane == 0) {
              uint8_t* dst = smem + OFF_Q + sl * TILE;
              const int row = p->row0 + (p->dual ? sl * a.tpt : 0);
              mbar_arrive_expect_tx(&q_full[sl], q_bytes);
              tma_load_3d(dst, &tmQ, &q_full[sl], 0, p->h * a.G, row);
              tma_load_3d(dst + HALF, &tmQ, &q_full[sl], 64, p->h * a.G, row);
            }
          }
          if (!ok) break;
        }
        // the piece before: rows of its last V tile from the sequence's last key to the next multiple of 16
        if (had) {
          if (before->tail()) {
            // loads before that tile: every K and V before it, its own K, and the first K of the next piece
            // if it came before slot 1's V
            const int st = (2 * (tiles - 1) + 1 + (!before->dual && !(before->tiles() & 1) && more ? 1 : 0)) % ST;
            ok = wait_for(&land[st], (n_land >> st) & 1u);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            n_land ^= 1u << st;
            uint8_t* vt = smem + OFF_RING + st * TILE;
            const int r0 = before->keys() - (before->nt - 1) * KT, r1 = (r0 + 15) & ~15;
            for (int r = r0 + (lane >> 4); r < r1; r += 2) {
              const int ch = lane & 15;
              *reinterpret_cast<uint4*>(vt + (ch >> 3) * HALF + sw128_off(r, (ch & 7) * 8)) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[st]);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&taken[(k + PR - 1) % PR]);
        }
        had = more;
        if (more) tiles += p->tiles();
      }
      if (!ok) set_status(a.status, 0x731u);
      if (!ok && lane == 0)                  // gave up: see the Q copies land before leaving
        for (int sl = 0; sl < 2; ++sl)
          if (n_q[sl] > 0) wait_for(&q_full[sl], (n_q[sl] - 1) & 1);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_SOFTMAX));
    // ------------------------------------------------------------ softmax and epilogue of slot sl
    const int sl = warp >> 2, row = tid & 127;
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + (uint32_t)sl * KT + lanes, t_o = tmem + 2 * KT + (uint32_t)sl * D + lanes;
    const int row_tok = row / a.G, row_head = row - row_tok * a.G;
    const bool row_used = row_tok < a.tpt;
    uint32_t n_s = 0, n_pair = 0, ph_o = 0;     // (ph_o: a phase bit per slot)
    bool ok = true;
    // A warp's rows of a piece, at its end: all dims of its slot's row tile (dual), or its slot's half of the dims
    // of the one row tile.  (Loops that run once in a while are kept short: unrolled, their instructions
    // came from L2 each time.)
    struct Rows {
      bool used;
      int c_lo, c_hi, c_first;             // dims; the CTA that opened the item
      uint16_t* out;
      float *part_o;                       // of CTA 0, slot 0
      float2* part_ml;
      unsigned *arrived, *taken;           // of a shared item (nullptr otherwise)
    };
    const int me = blockIdx.x;
    Shares shares{0, 0};
    auto rows_of = [&](const Piece& p) {
      Rows r;
      const int x = p.dual ? sl : 0, tok = x * a.tpt + row_tok, prow = x * TM + row;
      r.used = row_used && tok < p.tok;
      r.c_lo = p.dual ? 0 : sl * 64;
      r.c_hi = p.dual ? D : sl * 64 + 64;
      r.out = a.O + (size_t)(p.row0 + tok) * a.ldo + (size_t)(p.h * a.G + row_head) * D;
      // pieces in the workspace are [dim / 4][row][4]: consecutive rows in consecutive 16 bytes
      r.part_o = a.part_o + prow * 4;
      r.part_ml = a.part_ml + sl * (2 * TM) + prow;
      r.c_first = me;
      r.arrived = r.taken = nullptr;
      if (p.t0 > 0 || p.t1 < p.nt) {
        // the last CTA up to this one whose share does not start inside the item, 32 at a time
        for (unsigned out = 0; out == 0; r.c_first -= out ? __ffs(out) - 1 : 32)
          out = __ballot_sync(0xffffffffu, cut_tile(shares.start(max(r.c_first - lane, 0)) - p.start, p.dual,
                                                    p.keys(), p.nt) == 0);
        r.arrived = a.counters + 16 * r.c_first + warp;
        r.taken = r.arrived + 8;
      }
      return r;
    };
    auto part_at = [&](const Rows& r, int c) { return (size_t)c * 2 + (c == r.c_first ? 1 : 0); };
    auto store = [&](const Rows& r, int c, const float* v, float f, auto dims) {      // `dims` of them from c
      constexpr int N = decltype(dims)::value / 2;
      uint32_t w[N];
#pragma unroll
      for (int d = 0; d < N; ++d) w[d] = cvt_bf16x2(v[2 * d] * f, v[2 * d + 1] * f);
      if (!r.used) return;
      if (a.wide) {
#pragma unroll
        for (int d = 0; d < N; d += 8) st_global_32(r.out + c + 2 * d, w + d);
      } else {
#pragma unroll
        for (int d = 0; d < N; d += 4) st_global_16(r.out + c + 2 * d, w + d);
      }
    };
    // 32 unnormalised dims from c of this CTA's piece, from TMEM: O of the slot, or both slots' joined
    float fa = 1.f, fb = 0.f;
    bool have_b = false;
    auto own32 = [&](const Piece& p, int c, float* v) {
      tmem_ld_cols<32>(2 * KT + (p.dual ? (uint32_t)sl * D : 0u) + lanes + c, v);
      if (!p.dual) {
#pragma unroll
        for (int k = 0; k < 32; ++k) v[k] *= fa;
        if (have_b) {
          float w[32];
          tmem_ld_cols<32>(3 * KT + lanes + c, w);
#pragma unroll
          for (int k = 0; k < 32; ++k) v[k] += w[k] * fb;
        }
      }
    };
    // The CTAs that have a piece of an item: those of the first 32 from c_first on, and whether there are more.
    struct Sharers {
      unsigned has;
      int t;                               // tiles up to the last of the 32
    };
    auto sharers = [&](const Piece& p, int base, int t) {
      const int to = cut_tile(shares.start(base + lane + 1) - p.start, p.dual, p.keys(), p.nt);
      const int before = __shfl_up_sync(0xffffffffu, to, 1);
      Sharers s;
      s.has = __ballot_sync(0xffffffffu, to > (lane == 0 ? t : before));   // (a CTA without work has no piece)
      s.t = __shfl_sync(0xffffffffu, to, 31);
      return s;
    };
    // f(c) for batches of N sharers in CTA order (-1: none)
    auto batches = [&](const Piece& p, const Rows& r, const Sharers& first, auto n, auto&& f) {
      constexpr int BATCH = decltype(n)::value;
      Sharers s = first;
      for (int base = r.c_first;; base += 32) {
        while (s.has) {
          int c[BATCH];
#pragma unroll
          for (int k = 0; k < BATCH; ++k) {
            c[k] = s.has ? base + __ffs(s.has) - 1 : -1;
            s.has &= s.has - 1;
          }
          f(c);
        }
        if (s.t >= p.nt) break;
        s = sharers(p, base + 32, s.t);
      }
    };
    const Piece* shared_last = nullptr;    // the CTA's last piece, where its item goes on in the next CTA
    bool shared_first = false;             // the first piece's item came from the CTA before
    bool direct = false;                   // the last piece is joined from TMEM, with this maximum and sum
    float m_last = 0.f, l_last = 0.f;
    // Joins groups of dims of the pieces' rows, in CTA order whoever does it, as long as some are left to take (`here`:
    // all, with this CTA's piece from TMEM).  One pass over the pieces per group, their references and sums with
    // it (they mostly agree in the reference, so nothing is rescaled as a rule).  A few sharers take 32 dims at a
    // time and two pieces at once; many 16 and four, so that twice as many of them have a part and take fewer
    // rounds of loads (one token at 100000 keys of 8 heads on one kv head 37.4 -> 31.3 us, 64 rows of 16 heads at 60000
    // keys 42.2 -> 37.0; two sharers would lose 1 to 2 us to the smaller groups).
    auto join = [&](const Piece& p, const Rows& r, const Sharers& first, auto dims, auto batch, bool here) {
      constexpr int N = decltype(dims)::value, BATCH = decltype(batch)::value;
      const int groups = (r.c_hi - r.c_lo) / N;
      for (int g = 0;; ++g) {
        if (!here) {
          unsigned t = 0;
          if (lane == 0) t = atomicAdd(r.taken, 1u) & 0xffffu;
          g = (int)__shfl_sync(0xffffffffu, t, 0);
        }
        if (g >= groups) break;
        const int c0 = r.c_lo + N * g;
        float top = -INFINITY, sum = 0.f;
        float acc[N];
#pragma unroll
        for (int k = 0; k < N; ++k) acc[k] = 0.f;
        batches(p, r, first, batch, [&](const int (&c)[BATCH]) {
          float4 u[BATCH][N / 4];
          float2 ml[BATCH];
          float high = top;
#pragma unroll
          for (int k = 0; k < BATCH; ++k) {
            ml[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int d = 0; d < N / 4; ++d) u[k][d] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c[k] >= 0 && r.used && !(here && c[k] == me)) {
              ml[k] = __ldcg(r.part_ml + part_at(r, c[k]) * (4 * TM));
              const float* src = r.part_o + part_at(r, c[k]) * (2 * TM * D) + (size_t)(c0 >> 2) * (2 * TM * 4);
#pragma unroll
              for (int d = 0; d < N / 4; ++d)
                u[k][d] = __ldcg(reinterpret_cast<const float4*>(src + (size_t)d * (2 * TM * 4)));
            }
          }
          __syncwarp();
#pragma unroll
          for (int k = 0; k < BATCH; ++k) {
            if constexpr (N == 32)
              if (here && c[k] == me) {
                float v[32];
                own32(p, c0, v);
                ml[k] = make_float2(m_last, l_last);
#pragma unroll
                for (int d = 0; d < 8; ++d) u[k][d] = make_float4(v[4 * d], v[4 * d + 1], v[4 * d + 2], v[4 * d + 3]);
              }
            high = fmaxf(high, ml[k].x);
          }
          const float ref = high == -INFINITY ? 0.f : high;
          if (__any_sync(0xffffffffu, top != high)) {
            const float keep = ex2(top - ref);
            sum *= keep;
#pragma unroll
            for (int d = 0; d < N; ++d) acc[d] *= keep;
            top = high;
          }
#pragma unroll
          for (int k = 0; k < BATCH; ++k) {
            const float w = ex2(ml[k].x - ref);
            sum += ml[k].y * w;
#pragma unroll
            for (int d = 0; d < N / 4; ++d) {
              acc[4 * d] += u[k][d].x * w;
              acc[4 * d + 1] += u[k][d].y * w;
              acc[4 * d + 2] += u[k][d].z * w;
              acc[4 * d + 3] += u[k][d].w * w;
            }
          }
        });
        store(r, c0, acc, 1.f / sum, dims);
        __syncwarp();
      }
    };
    auto finish = [&](const Piece& p, float m, float l) {
      const Rows r = rows_of(p);
      // a piece of a shared item: how much of it has arrived by now (looked at while O is waited for)
      unsigned seen = 0;
      if (r.arrived && lane == 0) seen = ld_acquire(r.arrived);
      fa = 1.f;
      if (p.dual) {
        ok = ok && wait_for(&o_full[sl], (ph_o >> sl) & 1u);
        ph_o ^= 3u;
      } else {
        // the slots' sums joined
        have_b = p.tiles() > 1;            // (a piece of one tile leaves slot 1 out)
        ok = ok && wait_for(&o_full[0], ph_o & 1u);
        if (have_b) ok = ok && wait_for(&o_full[1], (ph_o >> 1) & 1u);
        ph_o ^= have_b ? 3u : 1u;
        s_ml[sl * TM + row] = make_float2(m, l);
        __syncwarp();
        uint64_t* both = pair + 2 * (warp & 3);
        if (lane == 0) mbar_arrive(both);
        ok = ok && wait_for(both, n_pair & 1);
        const float2 first = s_ml[row], second = s_ml[TM + row];
        m = fmaxf(first.x, second.x);
        const float base = m == -INFINITY ? 0.f : m;
        fa = ex2(first.x - base);
        fb = ex2(second.x - base);
        l = first.y * fa + second.y * fb;
      }
      __syncwarp();
      tc_fence_after();
      if (!r.arrived) {
        const float inv = 1.f / l;
#pragma unroll 1
        for (int c = r.c_lo; c < r.c_hi; c += 32) {
          float v[32];
          own32(p, c, v);
          store(r, c, v, inv, Int<32>{});
          __syncwarp();
        }
      } else {
        if (p.t0 > 0) shared_first = true;
        else shared_last = &p;             // (its entry of the ring is not posted again)
        // If all other pieces are there when the CTA that opened the item comes to its end, as a rule where two share
        // it, its piece need not go through memory.
        const Sharers all = sharers(p, r.c_first, 0);
        direct = p.t0 == 0 && all.t >= p.nt && __popc(all.has) == 2 &&
                 __shfl_sync(0xffffffffu, seen, 0) + (unsigned)p.tiles() == (unsigned)p.nt;
        m_last = m;
        l_last = l;
        if (!direct) {
          const size_t at = part_at(r, me);
#pragma unroll 1
          for (int c = r.c_lo; c < r.c_hi; c += 32) {
            float v[32];
            own32(p, c, v);
            float* dst = r.part_o + at * (2 * TM * D) + (size_t)(c >> 2) * (2 * TM * 4);
            if (r.used) {
#pragma unroll
              for (int d = 0; d < 32; d += 4)
                __stcg(reinterpret_cast<float4*>(dst + (size_t)(d >> 2) * (2 * TM * 4)),
                       make_float4(v[d], v[d + 1], v[d + 2], v[d + 3]));
            }
            __syncwarp();
          }
          if (r.used) __stcg(r.part_ml + at * (4 * TM), make_float2(m, l));
        }
        __syncwarp();
        if (lane == 0) {
          // (direct: nothing is left for the other sharer)
          if (direct) atomicAdd(r.taken, (unsigned)(r.c_hi - r.c_lo) >> 5);
          red_release(r.arrived, (unsigned)p.tiles());
        }
      }
      tc_fence_before();
      if (!p.dual) {
        __syncwarp();
        uint64_t* both = pair + 2 * (warp & 3) + 1;
        if (lane == 0) mbar_arrive(both);  // O and s_ml free again
        ok = ok && wait_for(both, n_pair & 1);
        ++n_pair;
      }
    };
    // At the CTA's end: the rows of a shared item are joined by the warps of all its CTAs that are still here when
    // the last piece arrives, a group of dims at a time.  A warp waits for that a while only: the warp that
    // brings the last piece joins whatever is left, so no CTA needs another one to run beside it.
    auto share = [&](const Piece& p, bool here) {
      const Rows r = rows_of(p);
      const Sharers all = sharers(p, r.c_first, 0);
      unsigned there = 0;
      if (lane == 0 && !here) {
        const uint64_t t0 = globaltimer();
        do {
          there = ld_acquire(r.arrived) == (unsigned)p.nt;
        } while (!there && globaltimer() - t0 < JOIN_WAIT_NS);
      }
      int n = __popc(all.has);
      Sharers s = all;
      for (int base = r.c_first; s.t < p.nt; n += __popc(s.has)) s = sharers(p, base += 32, s.t);
      if (here || __shfl_sync(0xffffffffu, there, 0)) {
        __syncwarp();
        if (__popc(all.has) > 4 || all.t < p.nt) join(p, r, all, Int<16>{}, Int<4>{}, false);
        else join(p, r, all, Int<32>{}, Int<2>{}, here);
      }
      // done with it; the last of the sharers clears their two words for the next launch
      if (lane == 0 && (int)(atomicAdd(r.taken, 0x10000u) >> 16) + 1 == n) {
        *r.taken = 0u;
        *r.arrived = 0u;
      }
      __syncwarp();
    };
    // (after a wait that ran out a warp stops waiting and leaves at its next piece)
    for (int k = 0; ok; ++k) {
      ok = wait_for(&posted[k % PR], (uint32_t)((k / PR) & 1));
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const Piece& p = ring[k % PR];
      if (k == 0) shares = *s_shares;
      if (!p.more) break;
      const bool dual = p.dual != 0;
      const int n = p.steps(sl), t0 = p.t0;
      const int x = dual ? sl : 0;         // the slot's row tile
      const int pos = p.pos + min(x * a.tpt + row_tok, p.tok - 1);      // the row sees keys 0 .. pos
      const bool live = row_used && x * a.tpt + row_tok < p.tok;        // (the other rows hold anything)
      const int pos_lo = __shfl_sync(0xffffffffu, pos, 0), pos_hi = __shfl_sync(0xffffffffu, pos, 31);
      // (a sequence's first row: one key, whose weight is then 1, which bf16 has exactly, whatever the score)
      const float scale = pos == 0 ? 1e-30f : a.scale_log2;
      float ref = 0.f, l_run = 0.f;
      for (int j = 0; j < n; ++j) {
        const int key0 = (t0 + (dual ? j : 2 * j + sl)) * KT;
        ok = ok && wait_for(&s_full[sl], n_s & 1);
        ++n_s;
        tc_fence_after();
        // hidden scores become -inf in place: the columns that some row of the warp does not see, 16 at a time
        // (a few of them only, and few instructions for what happens once per item)
        if (key0 + KT - 1 > pos_lo) {
          const int lim = pos - key0, hi = pos_hi - key0;
#pragma unroll 1
          for (int c = max(0, pos_lo + 1 - key0) & ~15; c < KT; c += 16) {
            uint32_t h[16];
            if (c <= hi) tmem_ld_cols16(t_s + c, h);
#pragma unroll
            for (int k = 0; k < 16; ++k)
              if (c + k > lim) h[k] = 0xff800000u;        // -inf
            tmem_st_cols16(t_s + c, h);
          }
          tmem_st_wait();
        }
        // Weights relative to the row's reference: the maximum of the first tile in which it sees a key, whose own weight
        // is then 1, exactly.  (bf16 weights are off by 1.7e-3 each in rms; a reference that is no maximum leaves that
        // to the largest weight too: rows of 16 keys 2.3e-3 off instead of 1.85e-3, of 128 keys 2.35e-3 instead of
        // 1.9e-3, logits of a few units; and scores far below a reference of 0 take small values out of fp32's range.
        // Looking costs 1 to 3 % on short prompts: 8 of 500 rows 27.2 -> 28.1 us, of 100 to 1900 rows 39.5 -> 40.4.)
        // Later tiles keep it, so that they need not wait for a maximum: any reference down to 2^20 below
        // the maximum gives the same quotients (bf16 and fp32 have exponents to spare, with values up to 1e25).
        // The tile's sum tells when it is out of that range; then the maximum is taken, O rescaled, and the weights
        // formed again.
        uint32_t pk[64];
        float tile_sum;
        for (bool look = __any_sync(0xffffffffu, live && l_run == 0.f);; look = true) {
          if (look) {
            float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
            for (int c = 0; c < KT; c += 64) {
              float v[64];
              tmem_ld_cols<64>(t_s + c, v);
#pragma unroll
              for (int k = 0; k < 64; ++k) top[k & 3] = fmaxf(top[k & 3], v[k]);
            }
            const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * scale;
            // (a sum above 2^27 has a weight above 2^20; nothing in sight: the reference stays)
            const bool move = l_run == 0.f ? mx > -INFINITY : mx > ref + 19.f;
            const float alpha = move && l_run != 0.f ? ex2(ref - mx) : 1.f;
            if (move) ref = mx;
            l_run *= alpha;
            // O is whole here: the scores' barrier came after the slot's P V before them
            if (__any_sync(0xffffffffu, live && alpha != 1.f)) {
#pragma unroll 1
              for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                tmem_ld_cols32(t_o + c, o);
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
                tmem_st_cols32(t_o + c, o);
              }
            }
          }
          uint32_t r[128];
          tmem_ld_cols128(t_s, r);
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          const float2 sc2 = make_float2(scale, scale), nb2 = make_float2(-ref, -ref);
#pragma unroll
          for (int k = 0; k < 64; ++k) {
            float2 e = fma2(make_float2(__uint_as_float(r[2 * k]), __uint_as_float(r[2 * k + 1])), sc2, nb2);
            e.x = ex2(e.x);
            e.y = ex2(e.y);
            sum[k & 1] = add2(sum[k & 1], e);
            pk[k] = cvt_bf16x2(e.x, e.y);
          }
          const float2 s2 = add2(sum[0], sum[1]);
          tile_sum = s2.x + s2.y;
          if (look || !__any_sync(0xffffffffu, live && !(tile_sum <= 0x1p27f))) break;
        }
        l_run += tile_sum;
        tmem_st_cols32(t_s, pk);
        tmem_st_cols32(t_s + 32, pk + 32);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[sl]);
      }
      finish(p, l_run == 0.f ? -INFINITY : ref, l_run);          // (no key in sight: no say in the reference)
      __syncwarp();
      if (lane == 0) mbar_arrive(&taken[k % PR]);
    }
    if (!ok) set_status(a.status, 0x741u);
    ok = __all_sync(0xffffffffu, ok);
#pragma unroll 1
    for (int k = 0; k < 2; ++k)
      if (ok && (k ? shared_first : shared_last != nullptr)) share(k ? *s_first : *shared_last, !k && direct);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

}  // namespace

cudaError_t launch_chunk_attention(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                   const ChunkAttnArgs& a, int grid, cudaStream_t s) {
  static bool configured[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !configured[dev]) {
    cudaError_t e = cudaFuncSetAttribute(chunk_attention_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != cudaSuccess) return e;
    // the split of registers between the warpgroups draws on what the launch has
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, chunk_attention_kernel);
    if (e != cudaSuccess) return e;
    if (fa.numRegs < REGS_ALL) return cudaErrorLaunchOutOfResources;
    if (dev >= 0 && dev < 64) configured[dev] = true;
  }
  cudaError_t e = launch_k(chunk_attention_kernel, dim3(grid), dim3(THREADS), SMEM, s, tq, tk, tv, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace spec
