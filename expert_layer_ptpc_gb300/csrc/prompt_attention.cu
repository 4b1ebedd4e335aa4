// Attention of many new tokens per context over the paged key-value cache.
//
//   s_ij = scale q_i . k_j for the tokens j that row i sees,
//   out_i = sum_j softmax(s_i)_j v_j,  lse_i = ln sum_j exp(s_ij)
//
// One pass over the tokens. The query heads of a kv head are rows of one matrix: row r of
// a context is head r % group of its new token r / group, so that 128 rows are full
// whatever the group. A CTA takes up to 256 rows (128 of 256 elements) against tiles of
// 128 tokens (64):
//   S = Q K^T (tcgen05, fp32 in TMEM);  x_j = s_j c,  w_j = 2^(x_j + F - M);
//   l += 2^-F sum_j w_j;  O += W V' (tcgen05, W from TMEM), V' = 2^-F V;  out = O / l,
// with c the factor of the row and tile, F the exponent that brings the tile's values
// into fp16, and M near the largest x + F so far: it is set 7 below a tile's largest, and
// moves only when a later one passes it by 15 (fp16 ends at 2^16), so that O is
// rarely rescaled. A weight is off by up to 2^-11 of it in fp16, or 2^-32 of the largest
// where that is more.
//
// What the tensor cores multiply: e4m3 codes in fp16, which holds them; a page's scale goes
// into them, relative to the tile's largest, brought to 2^6 (exact where it is a power of two,
// as the framework's writes make it, else a rounding to 11 bits of the scale and one of the
// product; codes go down to 2^-9 and fp16 to 2^-24, so that all is exact down to 2^-21 of
// the largest, off by up to 2^-31 of it below, and 0 from 2^-31 on; the largest is over all
// tokens that the item loads, whether a row sees them or not), a token's scale, relative to the
// largest too, into the score's column (keys) or, rounded to fp16, into the value. q in fp16,
// scaled by a power of two that brings its head's largest element into [2^8, 2^9): exact down
// to 2^-25 of that, below that off by up to 2^-33. A bf16 cache: q, k and v as they are, the weights rounded to
// bf16 (8 bits): the values' own products have no more, and a second product for the
// rest of a weight would cost half as much again.
//
// Roles of a CTA's warps: 0-3 and 4-7 the softmax of 128 rows each, a row a thread, and
// the rows' q; 8-11 fetch keys from the pages and lay them out for the tensor cores, 12-15
// values; 16 issues the products, 17 hands out the work. While one half's softmax runs, the
// other half's products do. (In a cut item of up to 128 rows the halves take every other tile of
// the same rows.) Loading warps turn codes into fp16 in registers: a lane asks for
// a piece of the next tile as it lays the last one's out, and the rows of the three tiles after
// that are on their way to L2. (Copies straight into shared memory, with the codes turned
// there, would pass 32 KB a tile more through it, which the products' operands already fill
// three quarters of the time that the products take.)
//
// The work is split over the CTAs by length: every item (a context's rows of one kv head)
// is given a weight, and every CTA an equal run of the weights' sum, whatever the
// lengths (they are read on the device). An item that several CTAs share leaves partial results,
// which a second kernel joins.
//
// GB300, 64 heads on 4 of 128 elements, a scale a page: a prompt of 8192 tokens 1015 us, 1.08
// PFLOP/s of cuBLAS's 1.95; 2048 tokens over 40001 with a scale a token 2.75 ms, 0.95 PFLOP/s;
// 5 tokens of each of 32 requests over up to 16384 (272 MB) 122 us, 2.2 TB/s, which the loading
// warps bound (2800 cycles a tile). The tensor
// pipe is 47% busy; what bounds it is the turn of a half: its softmax (about 2500 cycles a
// tile, of 512 that the exponentials take: loads from TMEM and issue slots shared with the
// loading warps) and then its two products, which one thread issues in some 1100. Tried
// beside it: tiles of 64 tokens with two of scores a half in TMEM, so that the softmax
// never waits for scores (1339 us against 1087: products of 64 columns cost as much to issue as
// those of 128); an issuing warp for each half (1236: the halves fall into step).
#include <algorithm>
#include <atomic>
#include <climits>

#include "attention.h"
#include "common.cuh"
#include "internal.h"
#include "tmem.cuh"

#include <cuda_fp16.h>

namespace moe {

namespace {

constexpr int kWorkers = 152;              // CTAs, one an SM
constexpr int kSoftWarps = 8;
constexpr int kLoadWarp0 = kSoftWarps;
constexpr int kLoadWarps = 4;              // of keys, and of values
constexpr int kMmaWarp = kLoadWarp0 + 2 * kLoadWarps;
constexpr int kPlanWarp = kMmaWarp + 1;
constexpr int kThreads = 32 * (kMmaWarp + 4);
// Registers of a thread, by role (640 threads are launched with 96 each: 61440).
constexpr int kSoftRegs = 136, kLoadRegs = 80, kMmaRegs = 48;
static_assert(256 * kSoftRegs + 256 * kLoadRegs + 128 * kMmaRegs <= 96 * kThreads, "registers");
constexpr int kAhead = 3;                  // tiles whose rows are on their way to L2
constexpr int kRing = 16;                  // segments handed out at a time
constexpr int kSides = 8;                  // tiles whose masks and factors are at hand
constexpr int kRequests = 256;             // contexts whose places a CTA keeps at hand
constexpr float kMostWeight = 15.0f;       // log2 of the largest weight let stand,
constexpr float kNewWeight = 7.0f;         // and of a tile's largest when M is set by it
// What an item costs beside its tiles, in tiles of 128 tokens: 48 short items of a window (the
// packed prompts) take 164 us with 2, 168 with 4 and 176 with 8, drafts 147, 121 and 117, 32 ragged
// chunks of up to 100 tokens 211, 164 and 162. And the least that a CTA is given: 4 tokens over
// 16384 take 67 us with 2, 68 with 4 and 50 with 8 (fewer pieces to join), four chunks of 40
// tokens 34, 39 and 47, nine short prompts 40, 39 and 48.
constexpr int kItemCost = 4;
constexpr int kLeastWork = 4;
// What a wait is given, beside kWaitLimitNs, for each 128 tokens of the longest run that a
// CTA can have: its halves can be a ring of segments apart, so that one waits for most of the
// run (2 to 3 us each).
constexpr double kWaitNsOfTile = 20000.0;
constexpr double kMostWaitNs = 1e11;

constexpr int kLeastExponent = -64;        // E and F as of scales of 2^-64 at least (sums end at 2^128)

enum Kind { kPageScales = 0, kTokenScales = 1, kBf16 = 2 };
enum Mode { kOne = 0, kTilesEach = 1, kRowsEach = 2 };
// Tiles of a segment whose halves share them out: drafts take 121 us with 2 and 4 and 125 with 8,
// 4 tokens over 16384 68, 68 and 58, four chunks of 40 tokens 40, 39 and 37.
constexpr int kLeastTiles = 4;

struct Args {
  CacheView c;
  const uint16_t* q;
  int64_t q_stride, out_stride;
  int rows, q_heads, batch, group;
  const int32_t *offsets, *lengths;
  float scale;
  int window;
  uint16_t* out;
  float* lse;
  struct Record* records;   // [kWorkers]
  float2* stats;            // [2 kWorkers][rows of an item] (M, l)
  float* parts;             // [2 kWorkers][D / 4][rows of an item][4]
  unsigned* err;
  unsigned long long wait_ns;   // after which a wait has run out
};

// What a CTA left of items that it shares with others: of its first one, begun by an
// earlier CTA (in slot 2 worker), and of its last one, which it began (slot 2 worker + 1).
struct Record {
  int4 head;                // context (-1: none), kv head, tile
  int4 tail;
  int token0, row0, rows;   // of the tail's rows: the first token of the context, first row, number
  int some;                 // whether the CTA had anything to do
};

template <int KIND, int D>
struct Shape {
  static constexpr int kStreams = D == 256 ? 1 : 2;       // of 128 rows
  static constexpr int kRows = 128 * kStreams;            // of an item
  static constexpr int kTile = D == 256 ? 64 : 128;       // tokens of a tile
  static constexpr int kStages = D == 64 ? 3 : 2;
  static constexpr int kQBytes = 128 * D * 2;             // of a stream
  static constexpr int kTileBytes = kTile * D * 2;
  // TMEM: tiles of scores, one a stream, or two in turn where there is one stream; then O. A
  // tile's weights lie in the second half of its scores.
  static constexpr int kSlots = 2 / kStreams;
  static constexpr int kSOut = 2 * kTile;
  static constexpr int kPOut = kTile / 2;
  static constexpr int kCols = 512;
  static constexpr int kSmemBytes = 1024 + kStreams * kQBytes + 2 * kStages * kTileBytes;
  static_assert(kSOut + kStreams * D <= kCols, "tensor memory");
};

// A context's rows: place of its first new token, rows and items of a kv head.
struct Context {
  int token0;      // row of q of its first new token
  int place;       // that token's place in the context (negative: before it)
  int rows;        // new tokens x group
  int items;
};
// An item, or a part of one: units [u0, u1) of `units` tiles.
struct Segment {
  int b, kv, item;
  int token0, place, row0, rows;   // rows [row0, row0 + rows) of the context
  int begin, end, start;           // tokens that take part; the first tile's first
  int u0, u1, units;
  __device__ __forceinline__ bool whole() const { return u0 == 0 && u1 == units; }
};

// Where a warp is in its CTA's run: the next place, and the run's end.
struct Walk {
  int b, kv, item, unit;
  int end[4];
  Context c;         // of context b
};

// A tile's masks and factors.
struct Side {
  uint32_t mask[4];      // which tokens are there: those of a loading warp each
  float key_up;          // 2^E
  float value_exp;       // F
};

struct Shared {
  uint64_t k_full[3], k_empty[3], v_full[3], v_empty[3];
  uint64_t q_full[2], s_full[2], p_full[2], o_full[2], o_empty[2];
  uint64_t maxed[2], drain, seg_full[kRing], seg_empty[kRing];
  uint32_t tmem;
  int abort;
  Side side[kSides];
  alignas(16) float key_scale[kSides][128];   // token scales times 2^-E, read as float4
  float row_scale[256];
  int maxima[2][2][kLoadWarps][2];   // of keys' loaders and values'
  int2 request[kRequests + 1];       // (first row, length)
  int64_t sums[kThreads / 32 + 1];
  int first;                         // the context of request[0]
  int place[2][4];                   // the run: first context, kv head, item, unit; and its end
  Segment ring[kRing];               // handed out and not yet done with; units < 0: no more
};

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(r))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)),
        "l"(reinterpret_cast<uint64_t&>(c)));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(r))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return r;
}
template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t w) {   // of the low two bytes
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)w));
  return h;
}
__device__ __forceinline__ uint32_t mul_f16(uint32_t a, uint32_t b) {
  const __half2 h = __hmul2(*reinterpret_cast<const __half2*>(&a),
                            *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&h);
}
// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float power(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
__device__ __forceinline__ int exponent(float x) {
  return (int)((__float_as_uint(x) >> 23) & 255u) - 127;
}

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void st_shared_16(uint32_t dst, uint32_t a, uint32_t b, uint32_t c,
                                             uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

// ---- the products ----
// Instruction descriptor of kind::f16, fp32 accumulator, 128 x N, B from rows along N
// (transposed) or along the contraction.
__host__ __device__ constexpr uint32_t idesc_f16(bool bf16, int n, bool b_rows_along_n) {
  return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) |
         ((b_rows_along_n ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | (8u << 24);
}
// Operand descriptors (smem_desc_k_sw128's fields) as a low word that counts with the address,
// and a constant high one: 8-row groups 1024 bytes apart, 128-byte swizzle. Rows along the
// contraction; or along the outer dimension (values: a row is 64 elements of one token), with
// the blocks of 64 elements `block` bytes apart.
constexpr uint32_t kDescHigh = (1024u >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_k(uint32_t saddr) { return saddr >> 4 | 1u << 16; }
__device__ __forceinline__ uint32_t desc_mn(uint32_t saddr, uint32_t block) {
  return saddr >> 4 | (block >> 4) << 16;
}
__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\t"
      "mov.b64 x, {%1, %5};\n\t"
      "mov.b64 y, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHigh)
      : "memory");
}
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\t"
      "mov.b64 y, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHigh)
      : "memory");
}
// One lane of a whole warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t yes;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(yes));
  return yes != 0;
}
// The same value in every lane, so that the compiler knows it.
__device__ __forceinline__ uint32_t uniform(uint32_t v) {
  return __shfl_sync(0xffffffffu, v, 0);
}

// ---- the work ----
template <int ROWS>
__device__ __forceinline__ Context context_of(const Args& a, int2 from, int to) {
  Context c;
  const int n = from.x >= 0 && to >= from.x && to <= a.rows ? to - from.x : 0;
  c.token0 = from.x;
  c.place = max(from.y, 0) - n;
  c.rows = n * a.group;
  c.items = (c.rows + ROWS - 1) / ROWS;
  return c;
}

// Weights of a context's items, in (tiles of 128 tokens) x group: item i has
//   min(a + s (i + 1), cap) + cost,  s the streams, a the tokens before its first new one.
struct Weights {
  int64_t a, cap, cost;
  int s;
  __device__ __forceinline__ int64_t of(int i) const {
    return min(a + (int64_t)s * (i + 1), cap) + cost;
  }
  __device__ __forceinline__ int64_t before(int64_t i) const {   // of items 0 .. i - 1
    const int64_t under = max((int64_t)0, min(i, (cap - a + s - 1) / s - 1));
    return under * a + s * (under * (under + 1) / 2) + (i - under) * cap + i * cost;
  }
};
template <int STREAMS>
__device__ __forceinline__ Weights weights_of(const Args& a, const Context& c) {
  Weights w;
  const int64_t room = (int64_t)a.c.max_pages << a.c.page_shift;
  w.a = (min((int64_t)max(c.place, 0), room) * a.group) >> 7;
  w.cap = a.window > 0 ? (((int64_t)a.window * a.group) >> 7) + STREAMS : (int64_t)1 << 60;
  w.a = min(w.a, w.cap);
  w.cost = (int64_t)kItemCost * a.group;
  w.s = STREAMS;
  return w;
}

template <int ROWS, int TILE>
__device__ __forceinline__ Segment segment_of(const Args& a, const Context& c, int b, int kv,
                                              int item) {
  Segment s;
  s.b = b;
  s.kv = kv;
  s.item = item;
  s.token0 = c.token0;
  s.place = c.place;
  s.row0 = item * ROWS;
  s.rows = min(ROWS, c.rows - s.row0);
  // (a tile behind the last token stays within an int)
  const int64_t room = min((int64_t)a.c.max_pages << a.c.page_shift, (int64_t)INT_MAX - 255);
  const int first = s.row0 / a.group, last = (s.row0 + s.rows - 1) / a.group;
  s.end = (int)max(min((int64_t)c.place + last + 1, room), (int64_t)0);
  s.begin = a.window > 0 ? (int)max((int64_t)c.place + first + 1 - a.window, (int64_t)0) : 0;
  s.begin = min(s.begin, s.end);
  s.start = s.begin & ~(TILE - 1);
  s.units = s.end > s.begin ? (int)(((int64_t)s.end - s.start + TILE - 1) / TILE) : 0;
  s.u0 = 0;
  s.u1 = s.units;
  return s;
}

// Hands out a CTA's run of the work to a warp, segment by segment.
template <int ROWS, int TILE>
__device__ __forceinline__ bool next_of(const Args& a, const Shared& sh, Walk& w, Segment& s) {
  const int first = sh.first;
  for (;;) {
    const bool last = w.b == w.end[0] && w.kv == w.end[1] && w.item == w.end[2];
    if (w.b >= a.batch || (last && w.unit >= w.end[3])) return false;
    s = segment_of<ROWS, TILE>(a, w.c, w.b, w.kv, w.item);
    s.u0 = min(w.unit, s.units);
    if (last) s.u1 = min(w.end[3], s.units);
    w.unit = 0;
    if (last) {
      w.b = a.batch;
    } else if (++w.item >= w.c.items) {
      w.item = 0;
      if (++w.kv == a.c.heads) {
        w.kv = 0;
        do {
          if (++w.b >= a.batch) break;
          const int at = w.b - first;
          int2 from, to;
          if (at < kRequests) {
            from = sh.request[at];
            to = sh.request[at + 1];
          } else {
            from = make_int2(a.offsets[w.b], a.lengths[w.b]);
            to.x = a.offsets[w.b + 1];
          }
          w.c = context_of<ROWS>(a, from, to.x);
        } while (w.c.items == 0);
      }
    }
    if (s.u1 > s.u0 || s.units == 0) return true;
  }
}

// Bounded wait of a whole warp: the same answer in every lane.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, Shared& sh,
                                          const Args& a, unsigned code) {
  const uint32_t at = smem_u32(bar);
  if (__all_sync(0xffffffffu, mbar_try_wait(at, parity))) return true;
  const unsigned long long t0 = global_timer_ns();
  for (uint32_t spin = 0;; ++spin) {
    if (__all_sync(0xffffffffu, mbar_try_wait(at, parity))) return true;
    if ((spin & 63u) == 63u) {
      bool bail = *reinterpret_cast<volatile int*>(&sh.abort) != 0;
      if (lane_id() == 0 && !bail && global_timer_ns() - t0 > a.wait_ns) {   // (one tells all)
        *reinterpret_cast<volatile int*>(&sh.abort) = 1;
        atomicOr(a.err, code);
        bail = true;
      }
      if (__any_sync(0xffffffffu, bail)) return false;
    }
  }
}
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if (lane_id() == 0) mbar_arrive(smem_u32(bar));
}

template <int KIND, int D>
__global__ void __launch_bounds__(kThreads, 1) prompt_attention_kernel(const Args a) {
  using S = Shape<KIND, D>;
  constexpr int kRows = S::kRows, kTile = S::kTile;
  constexpr bool kIsBf16 = KIND == kBf16;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared sh;
  uint8_t* const smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t q_at = smem_u32(smem);
  const uint32_t k_at = q_at + S::kStreams * S::kQBytes;
  const uint32_t v_at = k_at + S::kStages * S::kTileBytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 3; ++i) {
      mbar_init(smem_u32(&sh.k_full[i]), kLoadWarps);
      mbar_init(smem_u32(&sh.k_empty[i]), 1);
      mbar_init(smem_u32(&sh.v_full[i]), kLoadWarps);
      mbar_init(smem_u32(&sh.v_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sh.s_full[i]), 1);
      mbar_init(smem_u32(&sh.p_full[i]), 4);
      mbar_init(smem_u32(&sh.q_full[i]), 4);
      mbar_init(smem_u32(&sh.o_full[i]), 1);
      mbar_init(smem_u32(&sh.o_empty[i]), 4);
    }
    for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&sh.maxed[i]), kLoadWarps);
    mbar_init(smem_u32(&sh.drain), 1);
    for (int i = 0; i < kRing; ++i) {
      mbar_init(smem_u32(&sh.seg_full[i]), 1);
      mbar_init(smem_u32(&sh.seg_empty[i]), 4 * S::kStreams + 2 * kLoadWarps + 1);
    }
    sh.abort = 0;
    sh.place[0][0] = sh.place[1][0] = a.batch;   // nothing to do
    fence_barrier_init();
  }
  if (warp == kMmaWarp) tmem_alloc(smem_u32(&sh.tmem), S::kCols);
  pdl_wait();
  pdl_launch_dependents();

  // ---- this CTA's run of the work ----
  const int worker = blockIdx.x;
  {
    // (contexts that fit are read once, the others where they are wanted)
    const bool few = a.batch <= kRequests;
    if (few) {
      for (int i = threadIdx.x; i <= a.batch; i += kThreads)
        sh.request[i] = make_int2(a.offsets[i], i < a.batch ? a.lengths[i] : 0);
      __syncthreads();
    }
    auto context = [&](int b) -> Context {
      if (few) return context_of<kRows>(a, sh.request[b], sh.request[b + 1].x);
      return context_of<kRows>(a, make_int2(a.offsets[b], a.lengths[b]), a.offsets[b + 1]);
    };
    auto total_of = [&](int b) -> int64_t {
      if (b >= a.batch) return 0;
      const Context c = context(b);
      return c.items == 0 ? 0 : weights_of<S::kStreams>(a, c).before(c.items) * a.c.heads;
    };
    // sum over the threads before this one, and over all
    auto scan = [&](int64_t mine, int64_t& all) -> int64_t {
      int64_t up = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, up, o);
        if (lane >= o) up += v;
      }
      __syncthreads();
      if (lane == 31) sh.sums[warp] = up;
      __syncthreads();
      all = 0;
      int64_t before = up - mine;
      for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += sh.sums[w];
        all += sh.sums[w];
      }
      return before;
    };
    int64_t total = 0, mine = total_of(threadIdx.x), before;
    if (a.batch <= kThreads) {
      before = scan(mine, total);
    } else {
      int64_t sum = 0;
      for (int b = threadIdx.x; b < a.batch; b += kThreads) sum += total_of(b);
      scan(sum, total);
    }
    const int64_t least = (int64_t)kLeastWork * a.group;
    const int64_t workers = min((int64_t)gridDim.x, max((int64_t)1, total / least));
    if (worker < workers && total > 0) {
      const int64_t cut[2] = {total * worker / workers, total * (worker + 1) / workers};
      int64_t done = 0;
      for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
        int64_t all;
        if (a.batch > kThreads) {
          mine = total_of(b0 + threadIdx.x);
          before = done + scan(mine, all);
          done += all;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int64_t past = cut[i] - before;
          if (past < 0 || past >= mine) continue;
          // place `past` of context b
          const int b = b0 + threadIdx.x;
          const Context c = context(b);
          const Weights w = weights_of<S::kStreams>(a, c);
          const int64_t each = w.before(c.items);
          const int kv = (int)min(past / each, (int64_t)a.c.heads - 1);
          const int64_t in = past - kv * each;
          int lo = 0, hi = c.items;     // before(lo) <= in < before(hi)
          while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (w.before(mid) <= in) lo = mid; else hi = mid;
          }
          const Segment s = segment_of<kRows, kTile>(a, c, b, kv, lo);
          const int64_t rest = in - w.before(lo) - w.cost, span = w.of(lo) - w.cost;
          sh.place[i][0] = b;
          sh.place[i][1] = kv;
          sh.place[i][2] = lo;
          sh.place[i][3] = rest <= 0 ? 0 : (int)min(rest * s.units / span, (int64_t)s.units);
        }
      }
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (a.batch > kRequests) {
    for (int i = threadIdx.x; i <= kRequests; i += kThreads) {
      const int b = sh.place[0][0] + i;
      if (b <= a.batch)
        sh.request[i] = make_int2(a.offsets[b], b < a.batch ? a.lengths[b] : 0);
    }
  }
  if (threadIdx.x == 0) {
    a.records[worker].head.x = -1;
    a.records[worker].tail.x = -1;
    a.records[worker].some = 0;
    sh.first = a.batch > kRequests ? sh.place[0][0] : 0;
  }
  __syncthreads();
  const uint32_t tmem = sh.tmem;
  // The segments, from the warp that hands them out: number n is there (false: the run has
  // ended, or a wait has run out) and, when a role is done with it, free.
  auto take = [&](int n) -> bool {
    return warp_wait(&sh.seg_full[n % kRing], (n / kRing) & 1, sh, a, kErrTimeoutSched) &&
           sh.ring[n % kRing].units >= 0;
  };
  auto release = [&](int n) { warp_arrive(&sh.seg_empty[n % kRing]); };
  // place of 16-byte unit u of row r in an operand with `rows` rows: blocks of 128 bytes a
  // row, swizzled
  auto place = [](uint32_t base, int rows, int r, int u) -> uint32_t {
    return base + (u >> 3) * (rows * 128) + r * 128 + (((u & 7) ^ (r & 7)) << 4);
  };
  // How the two halves work on a segment: each on rows of its own; on the same rows and
  // every other tile (joined like pieces of different CTAs, and therefore only where there are
  // such); or the first alone.
  auto mode_of = [&](const Segment& s) -> int {
    if (S::kStreams == 1) return kOne;
    if (s.rows > 128) return kRowsEach;
    return s.whole() || s.u1 - s.u0 < kLeastTiles ? kOne : kTilesEach;
  };

  if (warp < kSoftWarps) {
    // ---------------- softmax ----------------
    more_registers<kSoftRegs>();
    const int me = warp >> 2;                 // the stream of two, and the half of TMEM
    const int row = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;   // of TMEM
    uint32_t s_phase = 0u;                    // of the stream's tiles of scores: bits 0, 1
    uint32_t o_phase = 0u;
    int tile = 0;                             // of all tiles (sides), at the segment's start
    bool ok = true;
    // This half's rows of q, a warp the rows of its threads; the factor of each.
    auto load_q = [&](const Segment& s) {
      const int base = mode_of(s) == kRowsEach ? me * 128 : 0;   // of the item's rows
      constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;   // lanes of a row, rows of a load
      constexpr int kBatch = 8;                              // loads in flight
      const int u = lane % kLanes;
      const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u;
      const float scale = fabsf(a.scale) * 1.4426950408889634f;
      const int r0 = (warp & 3) * 32 + lane / kLanes;        // of the half
      int token = (s.row0 + base + r0) / a.group;
      int in = s.row0 + base + r0 - token * a.group;         // head of the group
      for (int i0 = 0; i0 < 32; i0 += kBatch * kAtOnce) {
        uint4 raw[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          raw[i] = make_uint4(0u, 0u, 0u, 0u);
          if (i * kAtOnce < 32 - i0) {
            if (base + r0 + i0 + i * kAtOnce < s.rows)
              raw[i] = *reinterpret_cast<const uint4*>(
                  a.q + (int64_t)(s.token0 + token) * a.q_stride +
                  (int64_t)(s.kv * a.group + in) * D + u * 8);
            in += kAtOnce;
            while (in >= a.group) {
              in -= a.group;
              ++token;
            }
          }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          if (i * kAtOnce >= 32 - i0) break;
          const int r = r0 + i0 + i * kAtOnce;
          uint32_t x[4] = {raw[i].x ^ flip, raw[i].y ^ flip, raw[i].z ^ flip, raw[i].w ^ flip};
          float factor = scale;
          if (!kIsBf16) {
            float top = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              top = fmaxf(top, fmaxf(fabsf(bf16_lo(x[j])), fabsf(bf16_hi(x[j]))));
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1)
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            // a power of two brings the head's largest element into [2^8, 2^9)
            const int e = min(max(exponent(top), -110), 126);
            const float down = power(-e), up = power(8);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              x[j] = pack_f16(bf16_lo(x[j]) * down * up, bf16_hi(x[j]) * down * up);
            factor *= power(e - 8);
          }
          st_shared_16(place(q_at + me * S::kQBytes, 128, r, u), x[0], x[1], x[2], x[3]);
          if (u == 0) sh.row_scale[me * 128 + r] = factor;
        }
      }
      fence_proxy_async_smem();
      warp_arrive(&sh.q_full[me]);
    };
    auto has_q = [&](const Segment& s) { return me == 0 || mode_of(s) != kOne; };
    int number = 0;
    bool running = me < S::kStreams && take(0);
    if (running && has_q(sh.ring[0])) load_q(sh.ring[0]);
    for (; ok && running; release(number++)) {
      const Segment& seg = sh.ring[number % kRing];
      const int mode = mode_of(seg), tiles = seg.u1 - seg.u0;
      const bool mine = me == 0 || mode != kOne, whole = seg.whole();
      const int base = mode == kRowsEach ? me * 128 : 0;       // of the item's rows
      const int tile0 = mode == kTilesEach ? me : 0, step = mode == kTilesEach ? 2 : 1;
      const int r = seg.row0 + base + row;                     // of the context
      const bool live = mine && base + row < seg.rows;
      const int token = r / a.group, head = seg.kv * a.group + (r - token * a.group);
      // tokens [lo, hi) are seen (rows behind the last take anything; a warp of such rows
      // only keeps step)
      const bool works = __any_sync(0xffffffffu, live);
      const int hi = live ? (int)min((int64_t)seg.place + token + 1, (int64_t)seg.end) : INT_MAX;
      const int lo = live && a.window > 0
                         ? (int)max((int64_t)seg.place + token + 1 - a.window, (int64_t)0) : 0;
      float top = -INFINITY, sum = 0.f;
      const uint32_t o_at = tmem + lanes + S::kSOut + me * D;
      if (mine) {
        const float factor = sh.row_scale[me * 128 + row];
        const int start = seg.start + seg.u0 * kTile;
        for (int i = tile0; ok && i < tiles; i += step) {
          const int turn = S::kSlots == 2 ? i & 1 : 0, slot = me + turn;
          const uint32_t s_at = tmem + lanes + slot * kTile;
          ok = warp_wait(&sh.s_full[slot], (s_phase >> turn) & 1u, sh, a,
                         kErrTimeoutEpilogue);
          if (!ok) break;
          s_phase ^= 1u << turn;
          // The last tile's products. With one tile of scores in TMEM, these came after them;
          // with two, they are waited for before O is touched, and before the barrier can get a
          // phase further.
          auto last_products = [&]() -> bool {
            return S::kSlots == 1 || i == tile0 ||
                   warp_wait(&sh.o_full[me], o_phase ^ 1u, sh, a, kErrTimeoutEpilogue);
          };
          if (!works) {
            ok = last_products();
            if (!ok) break;
            warp_arrive(&sh.p_full[slot]);
            if (S::kSlots == 2 || i + step >= tiles) o_phase ^= 1u;
            continue;
          }
          tc_fence_after_sync();
          const Side& side = sh.side[(tile + i) & (kSides - 1)];
          // (above 0, so that it leaves the -inf of a token that is not seen as it is)
          const float c = fmaxf(factor * side.key_up, 0x1p-120f), f = side.value_exp;
          // what this row sees of the tile
          const int first = start + i * kTile;
          constexpr int kBits = kTile / kLoadWarps;   // tokens of a mask
          constexpr uint32_t kAll = kBits == 32 ? 0xffffffffu : 0xffffu;
          const uint32_t there = side.mask[0] & side.mask[1] & side.mask[2] & side.mask[3];
          const bool clear =
              __all_sync(0xffffffffu, there == kAll && lo <= first && hi - first >= kTile);
          // 64 scores at a time: all for their maximum, the last of them kept, and then the
          // others again for the weights (128 would not fit the registers). What a row does not
          // see is put back as -inf, keys' own scales with them. (The loops stay
          // rolled: the roles' code has to fit the instruction caches.)
          float s[64], high = -INFINITY;
#pragma unroll 1
          for (int h = 0; h < kTile / 64; ++h) {
            float m = tmem_load_max(s_at + 64 * h, s);
            if (KIND == kTokenScales || __builtin_expect(!clear, 0)) {
              if (KIND == kTokenScales) {
                const float4* const scales = reinterpret_cast<const float4*>(
                    sh.key_scale[(tile + i) & (kSides - 1)] + 64 * h);
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                  const float4 v = scales[j];
                  s[4 * j] *= v.x;
                  s[4 * j + 1] *= v.y;
                  s[4 * j + 2] *= v.z;
                  s[4 * j + 3] *= v.w;
                }
              }
              if (!clear) {
#pragma unroll
                for (int w = 0; w < 64 / kBits; ++w) {
                  const int at = first + 64 * h + w * kBits;
                  const int from = min(max(lo - at, 0), kBits), to = min(max(hi - at, 0), kBits);
                  uint32_t bits = side.mask[h * (64 / kBits) + w];
                  bits &= to >= 32 ? 0xffffffffu : (1u << to) - 1u;
                  bits &= from >= 32 ? 0u : ~((1u << from) - 1u);
#pragma unroll
                  for (int j = 0; j < kBits; ++j)
                    if (!((bits >> j) & 1u)) s[w * kBits + j] = -INFINITY;
                }
              }
              float t[2] = {s[0], s[1]};
#pragma unroll
              for (int j = 2; j < 62; j += 4) {
                t[0] = max3(t[0], s[j], s[j + 1]);
                t[1] = max3(t[1], s[j + 2], s[j + 3]);
              }
              m = max3(fmaxf(t[0], t[1]), s[62], s[63]);
              if (h < kTile / 64 - 1) {
                tmem_store(s_at, s);
                tmem_store_wait();
              }
            }
            high = fmaxf(high, m);
          }
          const float z = fmaf(high, c, f);
          bool waited = false;
          if (__builtin_expect(__any_sync(0xffffffffu, z > top + kMostWeight), 0)) {
            const float next = fmaxf(top, z - kNewWeight);
            const float down = top == -INFINITY ? 0.f : exp2_approx(top - next);
            top = next;
            sum *= down;
            if (i > tile0) {
              ok = last_products();
              if (!ok) break;
              waited = true;
              tc_fence_after_sync();
#pragma unroll 1
              for (int j = 0; j < D / 32; ++j) {
                float o[32];
                tmem_load(o_at + 32 * j, o);
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] *= down;
                tmem_store(o_at + 32 * j, o);
              }
            }
          }
          const float by = f - (top == -INFINITY ? 0.f : top);
          const float2 c2 = make_float2(c, c), by2 = make_float2(by, by);
          float2 add[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
          for (int h = kTile / 64 - 1; h >= 0; --h) {
            if (h < kTile / 64 - 1) tmem_load(s_at, s);
            uint32_t p[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const float2 x = fma2(make_float2(s[2 * j], s[2 * j + 1]), c2, by2);
              const float2 w = make_float2(exp2_approx(x.x), exp2_approx(x.y));
              add[j & 1] = add2(add[j & 1], w);
              p[j] = kIsBf16 ? pack_bf16(w.x, w.y) : pack_f16(w.x, w.y);
            }
            // (behind the scores that are still to be read)
            tmem_store(s_at + S::kPOut + 32 * h, p);
          }
          sum = fmaf((add[0].x + add[1].x) + (add[0].y + add[1].y), exp2_approx(-f), sum);
          tmem_store_wait();
          tc_fence_before_sync();
          if (!waited) {
            ok = last_products();
            if (!ok) break;
          }
          warp_arrive(&sh.p_full[slot]);
          if (S::kSlots == 2 || i + step >= tiles) o_phase ^= 1u;   // (commits on o_full)
        }
        if (!ok) break;
      }
      // q of the next segment, behind the last scores of this one
      running = take(number + 1);
      if (running && has_q(sh.ring[(number + 1) % kRing])) load_q(sh.ring[(number + 1) % kRing]);
      if (mine) {
        // the last products (o_phase has moved past them)
        ok = warp_wait(&sh.o_full[me], o_phase ^ 1u, sh, a, kErrTimeoutEpilogue);
        if (!ok) break;
        tc_fence_after_sync();
      }
      tile += tiles;
      if (!mine) continue;
      const int64_t slot = 2 * worker + (seg.u0 == 0 ? 1 : 0);
      const float inv = sum == 0.f ? 0.f : 1.f / sum;   // (0: nothing seen; NaN stays)
      const int64_t to = (int64_t)(seg.token0 + token);
      uint16_t* const out = a.out + to * a.out_stride + (int64_t)head * D;
      float4* const part = reinterpret_cast<float4*>(a.parts) +
                           slot * (kRows * D / 4) + me * 128 + row;
#pragma unroll 1
      for (int j = 0; j < D / 32; ++j) {
        float o[32];
        __syncwarp();
        tmem_load(o_at + 32 * j, o);
        if (live && whole) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            *reinterpret_cast<uint4*>(out + 32 * j + 8 * k) =
                make_uint4(pack_bf16(o[8 * k] * inv, o[8 * k + 1] * inv),
                           pack_bf16(o[8 * k + 2] * inv, o[8 * k + 3] * inv),
                           pack_bf16(o[8 * k + 4] * inv, o[8 * k + 5] * inv),
                           pack_bf16(o[8 * k + 6] * inv, o[8 * k + 7] * inv));
        } else if (live) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            part[(8 * j + k) * kRows] =
                make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
        }
      }
      tc_fence_before_sync();
      warp_arrive(&sh.o_empty[me]);
      if (live) {
        if (!whole) {
          a.stats[slot * kRows + me * 128 + row] = make_float2(top, sum);
          if (S::kStreams == 2 && mode == kOne)   // (the other half's tiles: none)
            a.stats[slot * kRows + 128 + row] = make_float2(-INFINITY, 0.f);
        } else if (a.lse != nullptr)
          a.lse[to * a.q_heads + head] =
              sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
      }
      if (threadIdx.x == 0) {
        Record& rec = a.records[worker];
        rec.some = 1;
        if (whole) {
        } else if (seg.u0 > 0) {
          rec.head = make_int4(seg.b, seg.kv, seg.item, 0);
        } else {
          rec.tail = make_int4(seg.b, seg.kv, seg.item, 0);
          rec.token0 = seg.token0;
          rec.row0 = seg.row0;
          rec.rows = seg.rows;
        }
      }
    }
  } else if (warp < kMmaWarp) {
    // ---------------- keys, or values ----------------
    fewer_registers<kLoadRegs>();
    const bool keys = warp < kLoadWarp0 + kLoadWarps;
    const int w = (warp - kLoadWarp0) & (kLoadWarps - 1);
    constexpr int kMine = kTile / kLoadWarps;            // tokens of a warp
    constexpr int kRowBytes = D * (kIsBf16 ? 2 : 1);
    constexpr int kChunks = kRowBytes / 16;              // 16-byte pieces of a row
    constexpr int kAtOnce = 32 / kChunks;                // rows of one load
    constexpr int kLoads = kMine * kChunks / 32;         // of a lane, of a tile
    // The lane's piece of a row, and its row of those of one load. Codes become two pieces of
    // fp16 each, and a row two or more blocks: eight neighbouring lanes take the same half of
    // the pieces of a block in two rows, so that their stores use all banks.
    constexpr int kQuads = kChunks / 4;
    const int chunk = kIsBf16 ? lane % kChunks : (lane & 3) | ((lane >> 3) % kQuads) << 2;
    const int sub = kIsBf16 ? lane / kChunks : ((lane >> 2) & 1) + 2 * ((lane >> 3) / kQuads);
    const uint8_t* const cache = static_cast<const uint8_t*>(keys ? a.c.k : a.c.v) + chunk * 16;
    uint64_t* const full = keys ? sh.k_full : sh.v_full;
    uint64_t* const empty = keys ? sh.k_empty : sh.v_empty;
    const uint32_t stages = keys ? k_at : v_at;
    uint32_t phase = 1u;                                 // (the stages are empty at first)
    int stage = 0, tile = 0;
    // The next tile to ask for: its segment's context, kv head and tokens, the lane's token,
    // and the tiles left of the segment.
    const int32_t* row_of_table = nullptr;
    int kv = 0, left = 0;
    uint32_t begin = 0, end = 0, token = 0;
    bool more = true;
    int number = 0;
    auto open = [&]() {   // the next segment
      more = take(number);
      if (!more) return;
      const Segment& s = sh.ring[number % kRing];
      left = s.u1 - s.u0;
      row_of_table = a.c.table + s.b * a.c.table_stride;
      kv = s.kv;
      begin = s.begin;
      end = s.end;
      token = (uint32_t)s.start + (uint32_t)s.u0 * kTile + w * kMine + lane;
      release(number++);
    };
    auto look = [&]() -> int32_t {
      return more && lane < kMine && token >= begin && token < end
                 ? row_of_table[token >> a.c.page_shift]
                 : -1;
    };
    auto advance = [&]() {
      token += kTile;
      if (--left == 0) open();
    };
    // What is known of the tiles ahead: the table entry of one that is looked up, and the
    // lane's cache row (all ones for none) of the one before it, whose lines are
    // on their way to L2.
    constexpr uint32_t kNoRow = 0xffffffffu;
    int32_t entry = -1;
    uint32_t spot = 0;
    bool asked = false;
    auto ask = [&]() {
      asked = more;
      entry = look();
      spot = ((uint32_t)kv << a.c.page_shift) + (token & ((1u << a.c.page_shift) - 1u));
      if (more) advance();
    };
    auto resolve = [&]() -> uint32_t {
      if ((uint32_t)entry >= (uint32_t)a.c.pages) return kNoRow;
      const uint32_t row = (((uint32_t)entry * a.c.heads) << a.c.page_shift) + spot;
#pragma unroll
      for (int i = 0; i < (kRowBytes + 127) / 128; ++i)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(cache - chunk * 16 +
                                                      (uint64_t)row * kRowBytes + 128 * i));
      return row;
    };
    // the lane's pieces of the next tile to lay out, asked for as those before are laid out
    uint4 reg[kIsBf16 ? 1 : kLoads];
    auto fetch = [&](uint32_t rows, int i) -> uint4 {
      const uint32_t row = __shfl_sync(0xffffffffu, rows, i * kAtOnce + sub);
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (row != kNoRow) v = *reinterpret_cast<const uint4*>(cache + (uint64_t)row * kRowBytes);
      return v;
    };
    // scales of the lane's token: the keys' loaders need both (they tell the softmax)
    float ks = 0.f, vs = 0.f;
    auto ask_scales = [&](uint32_t row) {
      ks = vs = 0.f;
      if (!kIsBf16 && row != kNoRow) {
        if (keys) ks = a.c.k_scale[row >> a.c.scale_shift];
        vs = a.c.v_scale[row >> a.c.scale_shift];
      }
    };
    open();
    ask();
    bool running = asked, ok = true;
    uint32_t now = resolve();               // the lane's row of this tile
    ask();
    bool follows[kAhead];                   // and of the next ones
    uint32_t then[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      follows[i] = asked;
      then[i] = resolve();
      ask();
    }
    if (running && !kIsBf16) {              // (bf16 rows go straight to the stages)
#pragma unroll
      for (int i = 0; i < kLoads; ++i) reg[i] = fetch(now, i);
      ask_scales(now);
    }
    while (running) {
      // the tile's factors and masks
      const unsigned mask = __ballot_sync(0xffffffffu, now != kNoRow);
      uint32_t factor = 0u;
      int e = 0, f = 0;
      if (!kIsBf16) {
        const int none = -1000;
        const int ke = ks > 0.f ? max(exponent(ks), kLeastExponent) : none;
        const int ve = vs > 0.f ? max(exponent(vs), kLeastExponent) : none;
        const int ktop = __reduce_max_sync(0xffffffffu, ke);
        const int vtop = __reduce_max_sync(0xffffffffu, ve);
        int(&maxima)[kLoadWarps][2] = sh.maxima[keys ? 0 : 1][tile & 1];
        if (lane == 0) {
          maxima[w][0] = ktop;
          maxima[w][1] = vtop;
        }
        uint64_t* const maxed = &sh.maxed[keys ? 0 : 1];
        warp_arrive(maxed);
        ok = warp_wait(maxed, tile & 1, sh, a, kErrTimeoutProducer);
        if (!ok) break;
        e = f = none;
#pragma unroll
        for (int i = 0; i < kLoadWarps; ++i) {
          e = max(e, maxima[i][0]);
          f = max(f, maxima[i][1]);
        }
        // the largest codes (448) times what is left of the scales: below 2^15, or 2^16
        e = e == none ? 0 : e - 6;
        f = f == none ? 0 : f - 6;
        // (a scale of 0 and one of NaN stay what they are)
        const float x = keys ? (KIND == kTokenScales ? 1.f : ks * power(-e)) : vs * power(-f);
        const __half h = __float2half_rn(x);
        factor = KIND == kTokenScales
                     ? __float_as_uint(x)
                     : (uint32_t)*reinterpret_cast<const uint16_t*>(&h) * 0x10001u;
      }
      if (keys) {
        Side& side = sh.side[tile & (kSides - 1)];
        if (lane == 0) {
          side.mask[w] = mask;
          if (w == 0) {
            side.key_up = power(e);
            side.value_exp = (float)f;
          }
        }
        if (KIND == kTokenScales && lane < kMine)
          sh.key_scale[tile & (kSides - 1)][w * kMine + lane] = ks * power(-e);
      }

      const uint32_t to = stages + stage * S::kTileBytes;
      const uint32_t mine = now;
      running = follows[0];
      now = then[0];
      if (!kIsBf16) ask_scales(now);
#pragma unroll
      for (int i = 0; i + 1 < kAhead; ++i) {
        follows[i] = follows[i + 1];
        then[i] = then[i + 1];
      }
      follows[kAhead - 1] = asked;
      then[kAhead - 1] = resolve();
      ask();
      ok = warp_wait(&empty[stage], phase, sh, a, kErrTimeoutProducer);
      if (!ok) break;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int r = i * kAtOnce + sub, row = w * kMine + r;
        if (kIsBf16) {
          const uint32_t from = __shfl_sync(0xffffffffu, mine, r);
          cp_async_16(place(to, kTile, row, chunk),
                      cache + (from == kNoRow ? 0 : (uint64_t)from * kRowBytes),
                      from == kNoRow ? 0u : 16u);
        } else {
          const uint32_t up = __shfl_sync(0xffffffffu, factor, r);
          const uint32_t in[4] = {reg[i].x, reg[i].y, reg[i].z, reg[i].w};
          uint32_t h[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            h[j] = e4m3x2_to_f16(in[j >> 1] >> (16 * (j & 1)));
            if (KIND == kTokenScales) {
              const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
              h[j] = pack_f16(v.x * __uint_as_float(up), v.y * __uint_as_float(up));
            } else {
              h[j] = mul_f16(h[j], up);
            }
          }
          st_shared_16(place(to, kTile, row, 2 * chunk), h[0], h[1], h[2], h[3]);
          st_shared_16(place(to, kTile, row, 2 * chunk + 1), h[4], h[5], h[6], h[7]);
          reg[i] = fetch(now, i);
        }
      }
      if (kIsBf16) {
        asm volatile("cp.async.commit_group;" ::: "memory");
        asm volatile("cp.async.wait_group 0;" ::: "memory");
      }
      fence_proxy_async_smem();
      warp_arrive(&full[stage]);
      ++tile;
      if (++stage == S::kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
  } else {
    fewer_registers<kMmaRegs>();
    if (warp == kMmaWarp) {
      // ---------------- products ----------------
      // (One thread issues a product in about 50 cycles, whatever its size, and a wait or a
      // commit in 100 or so more: what it issues is kept to the least.)
      uint32_t k_phase = 0u, v_phase = 0u;
      uint32_t q_phase = 0u, p_phase = 0u, oe_phase = 3u;   // bits 0, 1 (O is free at first)
      int k_stage = 0, v_stage = 0;
      bool ok = true;
      constexpr uint32_t kQk = idesc_f16(kIsBf16, kTile, false), kPv = idesc_f16(kIsBf16, D, true);
      for (int number = 0; ok && take(number); ++number) {
        const int mode = mode_of(sh.ring[number % kRing]);
        const int tiles = sh.ring[number % kRing].u1 - sh.ring[number % kRing].u0;
        release(number);
        // Task t: the scores, then the weights' products, of a stream and a tile; two tasks
        // are under way where there are two tiles of scores for them.
        const int tasks = mode == kRowsEach ? 2 * tiles : tiles;
        const int ahead = mode == kOne && S::kSlots == 1 ? 1 : 2;
        auto stream_of = [&](int t) { return mode == kOne ? 0 : t & 1; };
        auto slot_of = [&](int t) { return S::kSlots == 2 ? t & 1 : stream_of(t); };
        auto begins = [&](int t) { return t < (mode == kOne ? 1 : 2); };            // its stream
        auto ends = [&](int t) { return t >= tasks - (mode == kOne ? 1 : 2); };
        auto opens = [&](int t) { return mode != kRowsEach || (t & 1) == 0; };       // its tile
        auto closes = [&](int t) { return mode != kRowsEach || (t & 1) == 1; };
        auto scores = [&](int t) -> bool {
          const int stream = stream_of(t), slot = slot_of(t);
          if (begins(t)) {   // the stream's rows of q
            if (!warp_wait(&sh.q_full[stream], (q_phase >> stream) & 1u, sh, a,
                           kErrTimeoutMma))
              return false;
            q_phase ^= 1u << stream;
          }
          if (opens(t) && !warp_wait(&sh.k_full[k_stage], k_phase, sh, a, kErrTimeoutMma))
            return false;
          tc_fence_after_sync();
          const uint32_t d = uniform(tmem + slot * kTile);
          const uint32_t qs = uniform(desc_k(q_at + stream * S::kQBytes));
          const uint32_t ks = uniform(desc_k(k_at + k_stage * S::kTileBytes));
          if (elect_one()) {
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
              mma_f16_ss(d, qs + ((j >> 2) * (128 * 128) + (j & 3) * 32) / 16,
                         ks + ((j >> 2) * (kTile * 128) + (j & 3) * 32) / 16, kQk, j > 0 ? 1u : 0u);
            mma_commit(smem_u32(&sh.s_full[slot]));
            if (closes(t)) mma_commit(smem_u32(&sh.k_empty[k_stage]));
          }
          __syncwarp();
          if (closes(t) && ++k_stage == S::kStages) {
            k_stage = 0;
            k_phase ^= 1u;
          }
          return true;
        };
        for (int t = 0; ok && t < min(tasks, ahead); ++t) ok = scores(t);
        for (int t = 0; ok && t < tasks; ++t) {
          const int stream = stream_of(t), slot = slot_of(t);
          if (begins(t)) {   // O: the last segment's has been read
            ok = warp_wait(&sh.o_empty[stream], (oe_phase >> stream) & 1u, sh, a,
                           kErrTimeoutMma);
            if (!ok) break;
            oe_phase ^= 1u << stream;
          }
          if (opens(t)) {
            ok = warp_wait(&sh.v_full[v_stage], v_phase, sh, a, kErrTimeoutMma);
            if (!ok) break;
          }
          ok = warp_wait(&sh.p_full[slot], (p_phase >> slot) & 1u, sh, a, kErrTimeoutMma);
          if (!ok) break;
          p_phase ^= 1u << slot;
          tc_fence_after_sync();
          const uint32_t d = uniform(tmem + S::kSOut + stream * D);
          const uint32_t p = uniform(tmem + slot * kTile + S::kPOut);
          const uint32_t vs = uniform(desc_mn(v_at + v_stage * S::kTileBytes, kTile * 128));
          const uint32_t more = uniform(begins(t) ? 0u : 1u);
          if (elect_one()) {
#pragma unroll
            for (int j = 0; j < kTile / 16; ++j)
              mma_f16_ts(d, p + 8 * j, vs + j * (2048 / 16), kPv, j > 0 ? 1u : more);
            if (S::kSlots == 2 || ends(t)) mma_commit(smem_u32(&sh.o_full[stream]));
            if (closes(t)) mma_commit(smem_u32(&sh.v_empty[v_stage]));
          }
          __syncwarp();
          if (closes(t) && ++v_stage == S::kStages) {
            v_stage = 0;
            v_phase ^= 1u;
          }
          if (t + ahead < tasks) ok = scores(t + ahead);
        }
      }
      // every product has ended before tensor memory and shared memory are given back
      if (elect_one()) mma_commit(smem_u32(&sh.drain));
      __syncwarp();
      volatile int no_abort = 0;
      mbar_wait_bounded(smem_u32(&sh.drain), 0, &no_abort, a.err, kErrTimeoutDrain);
    } else if (warp == kPlanWarp) {
      // ---------------- the work, segment by segment ----------------
      Walk walk;
      walk.b = sh.place[0][0];
      walk.kv = sh.place[0][1];
      walk.item = sh.place[0][2];
      walk.unit = sh.place[0][3];
#pragma unroll
      for (int i = 0; i < 4; ++i) walk.end[i] = sh.place[1][i];
      if (walk.b < a.batch)
        walk.c = context_of<kRows>(a, sh.request[walk.b - sh.first],
                                   sh.request[walk.b - sh.first + 1].x);
      bool more = true;
      for (int n = 0; more; ++n) {
        Segment s;
        while ((more = next_of<kRows, kTile>(a, sh, walk, s)) && s.units == 0) {
          // rows that see nothing (the others get segments with tiles only: the loading warps
          // look some tiles ahead, and must find them within the ring)
          for (int r = s.row0; r < s.row0 + s.rows; ++r) {
            const int token = r / a.group, head = s.kv * a.group + r - token * a.group;
            const int64_t to = (int64_t)(s.token0 + token);
            if (lane < D / 8)
              *reinterpret_cast<uint4*>(a.out + to * a.out_stride + (int64_t)head * D + 8 * lane) =
                  make_uint4(0u, 0u, 0u, 0u);
            if (lane == 0 && a.lse != nullptr) a.lse[to * a.q_heads + head] = -INFINITY;
          }
        }
        if (!more) s.units = -1;
        if (!warp_wait(&sh.seg_empty[n % kRing], ((n / kRing) & 1) ^ 1, sh, a,
                       kErrTimeoutSched))
          break;
        if (lane == 0) sh.ring[n % kRing] = s;
        warp_arrive(&sh.seg_full[n % kRing]);
      }
    }
  }
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == kMmaWarp) tmem_dealloc(tmem, S::kCols);
}

// Joins the pieces of the items that several CTAs share: the one that CTA blockIdx.x
// began, 32 of its rows a block, four elements of a row a thread at a time. PAD: before that, all
// threads together make the rows behind the last context's those that see nothing.
constexpr int kJoinThreads = 256;

template <int KIND, int D, bool PAD>
__global__ void __launch_bounds__(kJoinThreads) prompt_join_kernel(const Args a, int workers) {
  constexpr int kRows = Shape<KIND, D>::kRows;
  pdl_wait();
  if (PAD) {
    const int from = min(max(a.offsets[a.batch], 0), a.rows);
    const int per = a.q_heads * (D / 8);   // 16-byte units of a token
    const int64_t me = (int64_t)(blockIdx.y * gridDim.x + blockIdx.x) * kJoinThreads + threadIdx.x;
    const int64_t all = (int64_t)gridDim.x * gridDim.y * kJoinThreads;
    for (int64_t i = me; i < (int64_t)(a.rows - from) * per; i += all)
      *reinterpret_cast<uint4*>(a.out + (from + i / per) * a.out_stride + (i % per) * 8) =
          make_uint4(0u, 0u, 0u, 0u);
    if (a.lse != nullptr)
      for (int64_t i = (int64_t)from * a.q_heads + me; i < (int64_t)a.rows * a.q_heads; i += all)
        a.lse[i] = -INFINITY;
  }
  const int w = blockIdx.x;
  const Record rec = a.records[w];
  if (rec.tail.x < 0) return;
  // the slots of the pieces: CTA w's, and those of the CTAs after it that went on (one
  // between them can have got nothing)
  __shared__ int slots[kWorkers];
  __shared__ int count;
  // of a piece's row, over the joined sum; items of up to 128 rows have two pieces a slot,
  // those of the CTA's halves
  constexpr int kMostHalves = kRows == 256 ? 2 : 1;
  __shared__ float weight[kMostHalves * kWorkers][32];
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int n = 1;
    bool more = true;
    if (lane == 0) slots[0] = 2 * w + 1;
    for (int i0 = w + 1; more && i0 < workers; i0 += 32) {
      int4 h = make_int4(-1, 0, 0, 0);
      int some = 1;
      if (i0 + lane < workers) {
        h = a.records[i0 + lane].head;
        some = a.records[i0 + lane].some;
      }
      const bool piece = h.x == rec.tail.x && h.y == rec.tail.y && h.z == rec.tail.z;
      // those up to the first CTA that did something else
      const unsigned other = __ballot_sync(0xffffffffu, !piece && some != 0);
      const unsigned upto = other ? (1u << (__ffs(other) - 1)) - 1u : 0xffffffffu;
      const unsigned pieces = __ballot_sync(0xffffffffu, piece) & upto;
      if ((pieces >> lane) & 1u) slots[n + __popc(pieces & lanemask_lt())] = 2 * (i0 + lane);
      n += __popc(pieces);
      more = other == 0;
    }
    if (lane == 0) count = n;
  }
  __syncthreads();
  const int row = blockIdx.y * 32 + (threadIdx.x & 31);
  const int halves = kMostHalves == 2 && rec.rows <= 128 ? 2 : 1;
  const int pieces = count * halves;
  // row of a piece among all slots' rows
  auto place = [&](int i) -> int64_t {
    return (int64_t)slots[i / halves] * kRows + (i % halves) * 128 + row;
  };
  if (blockIdx.y * 32 >= rec.rows) return;
  if (threadIdx.x < 32) {
    float top = -INFINITY, sum = 0.f;
    for (int i = 0; i < pieces; ++i) {
      const float2 s = a.stats[place(i)];
      weight[i][threadIdx.x] = s.x;
      // (a sum is NaN where a score was, and stays so, whatever the maxima)
      const float next = fmaxf(top, s.x);
      sum = sum * (top == -INFINITY ? 0.f : exp2_approx(top - next)) +
            s.y * (s.x == -INFINITY ? 0.f : exp2_approx(s.x - next));
      top = next;
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    for (int i = 0; i < pieces; ++i) {
      const float m = weight[i][threadIdx.x];
      weight[i][threadIdx.x] = sum != sum        ? sum
                               : m == -INFINITY ? -1.f   // nothing seen, or no tiles: no rows
                                                : exp2_approx(m - top) * inv;
    }
    if (row < rec.rows && a.lse != nullptr) {
      const int r = rec.row0 + row, token = r / a.group;
      const int head = rec.tail.y * a.group + (r - token * a.group);
      a.lse[(int64_t)(rec.token0 + token) * a.q_heads + head] =
          sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
    }
  }
  __syncthreads();
  if (row >= rec.rows) return;
  const int r = rec.row0 + row, token = r / a.group;
  const int head = rec.tail.y * a.group + (r - token * a.group);
  uint16_t* const out = a.out + (int64_t)(rec.token0 + token) * a.out_stride + (int64_t)head * D;
  const float4* const parts = reinterpret_cast<const float4*>(a.parts);
  constexpr int kSteps = D / 4 / (kJoinThreads / 32);   // of a thread
  float4 o[kSteps];
#pragma unroll
  for (int k = 0; k < kSteps; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = 0; i < pieces; ++i) {
    const float by = weight[i][threadIdx.x & 31];
    if (by < 0.f) continue;
    const int64_t at = (int64_t)slots[i / halves] * (D / 4) * kRows + (i % halves) * 128 + row;
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const int d = (threadIdx.x >> 5) + k * (kJoinThreads / 32);
      const float4 v = parts[at + (int64_t)d * kRows];
      o[k].x = fmaf(v.x, by, o[k].x);
      o[k].y = fmaf(v.y, by, o[k].y);
      o[k].z = fmaf(v.z, by, o[k].z);
      o[k].w = fmaf(v.w, by, o[k].w);
    }
  }
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    const int d = (threadIdx.x >> 5) + k * (kJoinThreads / 32);
    *reinterpret_cast<uint2*>(out + 4 * d) =
        make_uint2(pack_bf16(o[k].x, o[k].y), pack_bf16(o[k].z, o[k].w));
  }
}

template <int KIND, int D>
int launch(const Args& a, bool pad, cudaStream_t stream) {
  using S = Shape<KIND, D>;
  // the opt-in to more than 48 KB of shared memory, once per device
  static std::atomic<uint64_t> opted{0};
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess) return -3;
  const uint64_t bit = uint64_t(1) << (device & 63);
  if ((opted.load(std::memory_order_relaxed) & bit) == 0 || device >= 64) {
    if (cudaFuncSetAttribute(prompt_attention_kernel<KIND, D>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             S::kSmemBytes) != cudaSuccess)
      return -3;
    opted.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaError_t e = launch_kernel(true, dim3(kWorkers), dim3(kThreads), S::kSmemBytes, stream,
                                prompt_attention_kernel<KIND, D>, a);
  if (e != cudaSuccess) return -3;
  e = launch_kernel(true, dim3(kWorkers, S::kRows / 32), dim3(kJoinThreads), 0, stream,
                    pad ? prompt_join_kernel<KIND, D, true> : prompt_join_kernel<KIND, D, false>, a,
                    kWorkers);
  return e == cudaSuccess ? 0 : -3;
}

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }
size_t item_rows(int head_dim) { return head_dim == 256 ? 128 : 256; }

}  // namespace

size_t prompt_attention_ws_bytes(int, int head_dim, int) {
  const size_t rows = 2 * kWorkers * item_rows(head_dim);
  return align256(kWorkers * sizeof(Record)) + rows * sizeof(float2) +
         rows * head_dim * sizeof(float);
}

int launch_prompt_attention(const CacheView& c, const uint16_t* q, int64_t q_stride, int rows,
                            int q_heads, const int32_t* offsets, const int32_t* lengths, int batch,
                            float scale, int window, uint16_t* out, int64_t out_stride, float* lse,
                            bool pad, void* ws, cudaStream_t stream) {
  const int group = q_heads / c.heads;
  // the weights' sum over all items, times the CTAs, stays within 64 bits (contexts that
  // overlap, which the contract rules out, could add up to 2^16 times as much)
  const double items = (double)rows * q_heads / 128 + (double)batch * c.heads;
  const double room = std::min<double>((double)c.max_pages * (1 << c.page_shift), 0x1p31);
  const double work = items * (room * group / 128 + (double)rows * group / 128 + 8.0 * group);
  if (work > 0x1p46) return -2;
  Args a{};
  a.wait_ns = kWaitLimitNs +
              (unsigned long long)std::min(work / group / kWorkers * kWaitNsOfTile, kMostWaitNs);
  a.c = c;
  a.q = q;
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.rows = rows;
  a.q_heads = q_heads;
  a.batch = batch;
  a.group = group;
  a.offsets = offsets;
  a.lengths = lengths;
  a.scale = scale;
  a.window = window;
  a.out = out;
  a.lse = lse;
  uint8_t* const p = static_cast<uint8_t*>(ws);
  const size_t records = align256(kWorkers * sizeof(Record));
  a.records = reinterpret_cast<Record*>(p);
  a.stats = reinterpret_cast<float2*>(p + records);
  a.parts = reinterpret_cast<float*>(p + records +
                                     2 * kWorkers * item_rows(c.head_dim) * sizeof(float2));
  a.err = device_error_word();
  if (a.err == nullptr) return -3;
  const int kind = !c.e4m3 ? kBf16 : c.scale_shift > 0 ? kPageScales : kTokenScales;
  if (c.head_dim == 64)
    return kind == kBf16         ? launch<kBf16, 64>(a, pad, stream)
           : kind == kPageScales ? launch<kPageScales, 64>(a, pad, stream)
                                 : launch<kTokenScales, 64>(a, pad, stream);
  if (c.head_dim == 128)
    return kind == kBf16         ? launch<kBf16, 128>(a, pad, stream)
           : kind == kPageScales ? launch<kPageScales, 128>(a, pad, stream)
                                 : launch<kTokenScales, 128>(a, pad, stream);
  return kind == kBf16         ? launch<kBf16, 256>(a, pad, stream)
         : kind == kPageScales ? launch<kPageScales, 256>(a, pad, stream)
                               : launch<kTokenScales, 256>(a, pad, stream);
}

}  // namespace moe
