// Attention of one new token per context over the paged key-value cache.
//
//   s_j = scale q . k_j,  p_j = exp(s_j) / sum_i exp(s_i),  out = sum_j p_j v_j,
//   lse = ln sum_j exp(s_j)
//
// One pass over the cached tokens. In base 2, with x_j = s_j log2(e) and an
// e4m3 value row v_j = a_j c_j (a_j its scale, c_j its codes), a warp keeps
//   M (near max_j x_j + log2 a_j),  w_j = 2^(x_j + log2 a_j - M),
//   acc = sum_j w_j c_j,   l = sum_j w_j / a_j,
// so that out = acc / l and lse = (M + log2 l) ln 2. The scale of a value row
// goes into its weight's exponent: the weights stay in fp16's range whatever
// the scales, and the codes go to the tensor cores unscaled. M is set 7 below a
// tile's maximum, and moves only when a later one passes it by 15 (fp16 ends at
// 2^16), so that the accumulators are rarely rescaled. A weight's rounding is off by up
// to 2^-11 of it, or by 2^-32 of the largest weight where that is more: weights below
// that are rounded to zero, and elements whose codes are zero in all heavier tokens
// lose what they would have added. The sum takes the weights unrounded; in it a weight
// vanishes below 2^-133 of the largest (fp32), so that tokens of equal p_j all
// count as long as their value scales are within 2^100 of one another. Sums
// and accumulators are fp32.
//
// The work is bound by the cache's bytes: 4 D flops a token and query head
// against 2 D + 8 bytes a token and kv head, 31 flop/byte with 16 query heads a
// kv head. Hence:
// * the length is split. The batch's contexts are cut into units of 64 or 128
//   tokens of one kv head, and every CTA gets an equal run of units, whatever the
//   lengths (they are read on the device, so a captured graph follows them). A
//   context that ends up on several CTAs leaves partial results, which a
//   second kernel joins.
// * the up to 16 query heads of a kv head are the rows of one m16n8k16 tensor
//   core tile; in larger calls up to 32 of 64 or 128 elements are two tiles, for
//   which a token is copied and converted once (64 contexts of 8000 tokens, 80 heads on
//   4, 128 elements: e4m3 124 us, bf16 172; as two work items 180 and 319). More heads
//   a kv head are further work items, which find the tokens in L2.
// * each warp has tiles of 16 or 32 tokens of its own in flight (cp.async),
//   kStages deep, with barriers of the warp only.
// * the order of the head's elements in the contraction is free (q is laid out
//   to match), so that a lane's operands of a key row are 16 neighbouring bytes:
//   word w of them feeds contraction step w. The order of the output's elements
//   is free too: a lane's operands of a value row are 16 neighbouring bytes,
//   byte j of them belongs to output tile j.
// e4m3 operands are converted to fp16, which holds every code. q goes from
// bf16 to fp16 scaled by a power of two per head, which brings the head's largest
// element into [1, 2): elements under 2^-17 lose bits of their 8 (fp16's smallest step
// is 2^-24), and are off by up to 2^-25. The weights are rounded to fp16 (11 bits). With
// a bf16 cache the operands are bf16, and the weights go in as the sum of two
// bf16 numbers (16 bits).
//
// A cache with one scale a page and head goes the same way: a token's scale is then read from
// its page's (128 contexts as below 174 us, 6.2 TB/s, for 8 bytes a token less).
//
// GB300: 128 contexts of 0 to 16384 tokens, 64 query heads on 4 of 128, e4m3 (1.11 GB):
// 183 us, 6.1 TB/s of the copy's 6.8; one context of 262143 tokens (277 MB): 54 us, of
// which 40 are the tiles at the copy's rate and the rest the first loads, the last CTA
// and the joining kernel. 8 warps an SM of up to 255 registers; the tensor cores are 30%
// busy, and the issue slots 40%.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "attention.h"
#include "common.cuh"
#include "internal.h"

#include <cuda_fp16.h>

namespace moe {

namespace {

constexpr int kSms = 152;
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kGroup = 16;                 // tokens of one tensor core contraction
constexpr int kMmaRows = 16;               // query heads of a tensor core tile
constexpr int kMaxCtasPerSm = 3;
constexpr int kMaxWorkers = kSms * kMaxCtasPerSm;
constexpr float kMostWeight = 15.0f;       // log2 of the largest weight let stand,
constexpr float kNewWeight = 7.0f;         // and of a tile's largest when M is set by it
// What an item of a context costs beside its units, in units: fetching q, and
// joining the warps. The work is cut with this included, or the workers that
// get many short contexts would be the last to finish.
constexpr uint32_t kItemCost = 2;
constexpr int kLengths = 256;              // contexts whose lengths a worker keeps at hand
// Contexts of at most so many units are not cut when a CTA can have each item:
// the second kernel is spared. (GB300, 64 heads of 128 on 4, 300 tokens, in a graph:
// 7.6 us against 8.0 us cut in three, and one launch less.)
constexpr int kWholeUnits = 4;

// An item that several workers share, and where they left its pieces: the first
// worker's in slot 2 first + 1, worker w's after it in slot 2 w.
struct Joint {
  int32_t item;     // of all the batch's
  int32_t first;    // the first worker
  int32_t pieces;   // number of workers; below 2: nothing to join
  int32_t pad;
};

struct Args {
  CacheView c;
  const uint16_t* q;
  int64_t q_stride;
  int batch, q_heads, group;   // group: query heads of a kv head
  int chunks;                  // items that a group is cut into
  int rows;                    // query heads of an item, at most
  const int32_t* lengths;
  float scale;
  int window;
  int whole;                   // a CTA takes one item, all of it
  uint16_t* out;
  float* lse;
  Joint* joints;               // [joint_count]: by item, or by the item's first worker
  int joint_count;             // the fewer of the two
  int by_worker;
  float2* stats;               // [slots][rows] (M, l)
  float* parts;                // [slots][rows][D]
};

// First and last tokens that take part, and the units (of `unit` tokens) they
// cover; the first unit starts at a multiple of kGroup.
struct Span {
  uint32_t begin, end, start, units;
};

__device__ __forceinline__ Span span_of(const Args& a, int length, int unit) {
  const int64_t room = (int64_t)a.c.max_pages << a.c.page_shift;
  Span s;
  s.end = (uint32_t)min((int64_t)max(length, 0), room);
  s.begin = a.window > 0 ? (uint32_t)max(max(length, 0) - a.window, 0) : 0u;
  s.start = s.begin & ~(uint32_t)(kGroup - 1);
  s.units = s.end > s.begin ? (s.end - s.start + unit - 1) / unit : 0u;
  return s;
}

// M: tensor core tiles of query heads an item has.
template <bool E4M3, int D, int M>
struct Shape {
  static constexpr int kRows = M * kMmaRows;                // query heads of an item
  static constexpr int kRowBytes = D * (E4M3 ? 1 : 2);
  static constexpr int kTile = kRowBytes <= 128 ? 32 : 16;  // tokens a warp takes at a time
  static constexpr int kUnit = kWarps * kTile;              // tokens of a work unit
  static constexpr int kGroups = kTile / kGroup;
  static constexpr int kKeyPieces = kRowBytes / 64;        // 16-byte pieces a lane holds of a key
  static constexpr int kChunk = E4M3 && D >= 128 ? 16 : 8; // elements of a value piece
  static constexpr int kPieceBytes = kChunk * (E4M3 ? 1 : 2);
  static constexpr int kValuePieces = D / 8 / kChunk;      // pieces a lane holds of a value
  static constexpr int kKeyBytes = kTile * kRowBytes;      // of a stage, and as much of values
  static constexpr int kCtas = kRowBytes == 64 && M == 1 ? 3 : kRowBytes == 512 ? 1 : 2;
  static constexpr int kStages = kRowBytes == 64 || kRowBytes == 512 ? 3 : 2;
  static constexpr int kSides = 4;                         // at least kStages + 1
  static constexpr int kScaleBytes = E4M3 ? kSides * kTile * 12 : 0;
  static constexpr int kStageBytes = 2 * kKeyBytes;
  static constexpr int kWarpBytes = kStages * kStageBytes + kScaleBytes;
  static constexpr int kJoinBytes = kRows * D * 4;         // an accumulator tile
  // q's operands: 64 registers with 256 elements or two tiles of 128, next to 128 of
  // accumulators. For two tiles and for e4m3 heads of 256 they are in shared memory, and
  // fetched when a segment begins instead of before (64 contexts of 8000 tokens, 16 heads
  // on 2 of 256 elements, e4m3: 101 us, 137 with them in registers; two tiles of 64: 82
  // us, 87). bf16 heads of 256 keep them in registers: their stages and joins take 224 KB,
  // and q's 8 do not fit beside them; the kernel moves 6.3 TB/s all the same. Kernels of 256 elements and
  // of two tiles of 128 spill 44 to 164 bytes at 255 registers; the others none.
  static constexpr bool kSharedQ = M == 2 || (E4M3 && D == 256);
  static constexpr int kQBytes = kSharedQ ? M * (D / 16) * 512 : 0;
  static constexpr int kSmemBytes = kWarps * kWarpBytes + 2 * kJoinBytes + kQBytes;
  // A tile's rows lie in shared memory as in the cache, except that within each
  // 128-byte line the 16-byte pieces are permuted: the number of a key's piece is
  // xored with 4 in odd rows (8 lanes read 4 pieces of two neighbouring rows), a
  // value's with row & 6 (8 lanes read 2 pieces of 4 rows two apart), 64-byte
  // keys excepted (two rows are a line). Written out as what depends on the lane,
  // once a kernel, and what the compiler knows.
  //
  // Writing: lane's piece 32 j + lane of a group of rows goes to byte
  // (lane part ^ step part) + 512 j.
  static __device__ __forceinline__ int key_write(int lane) {
    const int odd = kRowBytes == 128 ? (lane >> 3) & 1 : kRowBytes == 256 ? (lane >> 4) & 1 : 0;
    return (lane ^ (odd << 2)) * 16;
  }
  static __device__ __forceinline__ constexpr int key_write_step(int j) {
    return kRowBytes == 512 ? (j & 1) * 64 : 0;
  }
  static __device__ __forceinline__ int value_write(int lane) {
    const int key = kRowBytes == 64 ? (lane >> 2) & 6 : kRowBytes == 128 ? (lane >> 3) & 2 : 0;
    return (lane ^ key) * 16;
  }
  static __device__ __forceinline__ constexpr int value_write_step(int j) {
    // (a step is 512 / kRowBytes rows)
    return (j * (512 / kRowBytes) & 6 & (kRowBytes == 64 ? 0 : kRowBytes == 128 ? 4 : 6)) * 16;
  }
  // Reading: pieces 4 p + t of key row 8 n + g, at byte (lane part ^ (p odd ? 64 : 0))
  // + 128 (p / 2) + 8 n kRowBytes; the operands of value row 2 t + r, r = 0, 1, 8, 9, at
  // lane part + r kRowBytes + 128 p (64-byte rows: (lane part ^ (r odd ? 64 : 0)) +
  // (r & 8) kRowBytes).
  static __device__ __forceinline__ int key_read(int g, int t) {
    return ((g * (kRowBytes / 16) + t) ^ (kRowBytes == 64 ? 0 : (g & 1) << 2)) * 16;
  }
  static __device__ __forceinline__ int value_read(int g, int t) {
    return kRowBytes == 64 ? ((8 * t + (g >> 1)) ^ (2 * t)) * 16 + (g & 1) * 8
                           : 2 * t * kRowBytes + (g ^ (2 * t)) * 16;
  }
  static_assert(kCtas * (kSmemBytes + 1024 + 2048) <= 228 * 1024, "shared memory");
  static_assert(kCtas <= kMaxCtasPerSm, "workspace slots");
};

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// Copies `bytes` bytes and fills the rest of the piece with zeros.
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float log2_approx(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Four e4m3 codes of a word as two fp16 pairs.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// acc += A B, 16 x 8 x 16.
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

// Largest over the four lanes that share a row of the accumulator tile.
__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
__device__ __forceinline__ float quad_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  return v + __shfl_xor_sync(0xffffffffu, v, 2);
}

__device__ __forceinline__ float weight(float m, float top) {   // 2^(m - top), 0 for no tokens
  return m == -INFINITY ? 0.f : exp2_approx(m - top);
}

// Place of float4 f of a row of D floats in the join's shared memory: lanes
// that hold neighbouring pieces of the same or the next row fall into
// different banks.
template <int CHUNK>
__device__ __forceinline__ int join_place(int row, int f) {
  return CHUNK == 16 ? f ^ ((((f >> 3) & 3) << 1) | (row & 1))
                     : f ^ (((f >> 3) & 1) | ((row & 1) << 1));
}

// A worker's part of one item of one context: units [u0, u1) of the item, which
// ends at place `end` of the batch's work.
struct Segment {
  int b, kv, chunk;
  uint32_t u0, u1;
  Span span;
  uint32_t end;
  __device__ __forceinline__ bool whole() const { return u0 == 0 && u1 == span.units; }
};

// Hands out a worker's run of the batch's work, segment by segment. An item
// takes kItemCost + units places; a run that ends within the first of them
// gets nothing of it.
struct Walker {
  uint32_t place, stop;    // next place, and the run's end
  int b, kv, chunk;        // of the next place
  uint32_t in;             // places of the item before it
  Span span;

  __device__ __forceinline__ bool next(const Args& a, const int* lengths, int first, int unit,
                                       Segment& s) {
    while (place < stop) {
      const uint32_t size = kItemCost + span.units;
      const uint32_t to = min(size, in + (stop - place));
      s.b = b;
      s.kv = kv;
      s.chunk = chunk;
      s.span = span;
      s.u0 = max(in, kItemCost) - kItemCost;
      s.u1 = max(to, kItemCost) - kItemCost;
      s.end = place + (size - in);
      place += to - in;
      in = 0;
      if (place < stop && ++chunk == a.chunks) {
        chunk = 0;
        if (++kv == a.c.heads) {
          kv = 0;
          do {
            if (++b >= a.batch) {   // (lengths changed under the kernel)
              place = stop;
              break;
            }
            const int at = b - first;
            span = span_of(a, at < kLengths ? lengths[at] : a.lengths[b], unit);
          } while (span.units == 0);
        }
      }
      if (s.u1 > s.u0) return true;
    }
    return false;
  }
};

// out and lse of an item of a context without tokens.
__device__ __forceinline__ void zero_rows(const Args& a, int b, int item, int head_dim) {
  const int kv = item / a.chunks;
  const int head0 = kv * a.group + (item - kv * a.chunks) * a.rows;
  const int rows = min(a.rows, (kv + 1) * a.group - head0);
  const int64_t at = (int64_t)b * a.q_heads + head0;
  for (int i = threadIdx.x; i < rows * (head_dim / 8); i += kThreads)
    reinterpret_cast<uint4*>(a.out + at * head_dim)[i] = make_uint4(0u, 0u, 0u, 0u);
  if (a.lse != nullptr && threadIdx.x < rows) a.lse[at + threadIdx.x] = -INFINITY;
}

template <bool E4M3, int D, int M>
__global__ void __launch_bounds__(kThreads, Shape<E4M3, D, M>::kCtas)
    paged_attention_kernel(const Args a) {
  using S = Shape<E4M3, D, M>;
  constexpr int kRows = S::kRows;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float2 stats[2][kRows];
  __shared__ int lengths[kLengths];
  __shared__ Walker walkers[kWarps][2];   // a warp's: of the work, and of the copies
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;    // row (or column) and place in a tile's fragments
  uint8_t* const stage0 = smem + warp * S::kWarpBytes;
  const uint32_t stage_u32 = smem_u32(stage0);
  float* const side0 = reinterpret_cast<float*>(stage0 + S::kStages * S::kStageBytes);
  uint8_t* const join0 = smem + kWarps * S::kWarpBytes;
  pdl_wait();
  pdl_launch_dependents();

  // ---- this worker's run of the batch's work: places [lo, hi) ----
  const int items = a.c.heads * a.chunks;
  auto places_of = [&](int b) -> uint32_t {   // (all together fit: the host sees to it)
    const uint32_t units = b < a.batch ? span_of(a, a.lengths[b], S::kUnit).units : 0u;
    return units == 0 ? 0u : (units + kItemCost) * items;
  };
  uint32_t total = 0, workers = 1, lo = 0, hi = 0;
  const uint32_t worker = blockIdx.x;
  int first = 0;          // the context that place lo falls into
  uint32_t before = 0;    // places of the contexts before it
  if (a.whole) {
    first = blockIdx.x / items;
    const uint32_t size = places_of(first) / items;
    if (size == 0) {
      zero_rows(a, first, blockIdx.x - first * items, D);
      return;
    }
    lo = (blockIdx.x - first * items) * size;
    hi = lo + size;
  } else {
    for (int b = lane; b < a.batch; b += 32) total += places_of(b);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    for (int b = blockIdx.x; b < a.batch; b += gridDim.x)
      if (places_of(b) == 0)
        for (int item = 0; item < items; ++item) zero_rows(a, b, item, D);
    if (a.by_worker && threadIdx.x == 0) a.joints[worker].pieces = 0;
    workers = min(gridDim.x, total);
    if (worker >= workers) return;
    // worker w's run starts at floor(total w / workers)
    const uint32_t each = total / workers, over = total - each * workers;
    lo = each * worker + over * worker / workers;
    hi = each * (worker + 1) + over * (worker + 1) / workers;
    for (int b0 = 0;; b0 += 32) {
      if (b0 >= a.batch) return;   // (lengths changed under the kernel)
      const uint32_t mine = places_of(b0 + lane);
      uint32_t up = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, up, o);
        if (lane >= o) up += v;
      }
      const unsigned past = __ballot_sync(0xffffffffu, before + up > lo);
      if (past != 0) {
        const int in = __ffs(past) - 1;
        first = b0 + in;
        before += __shfl_sync(0xffffffffu, up - mine, in);
        break;
      }
      before += __shfl_sync(0xffffffffu, up, 31);
    }
    for (int i = threadIdx.x; i < kLengths; i += kThreads)
      lengths[i] = first + i < a.batch ? a.lengths[first + i] : 0;
    __syncthreads();
  }
  {
    Walker w;
    w.place = lo;
    w.stop = hi;
    w.b = first;
    w.span = span_of(a, a.lengths[first], S::kUnit);
    const uint32_t past = lo - before, size = kItemCost + w.span.units;
    const int item = past / size;
    w.kv = item / a.chunks;
    w.chunk = item - w.kv * a.chunks;
    w.in = past - item * size;
    if (w.kv >= a.c.heads) w.stop = lo;   // (as above)
    if (lane < 2) walkers[warp][lane] = w;
    __syncwarp();
  }
  // (in shared memory: they are wanted once a segment, and registers are scarce)
  auto next_segment = [&](int which, Segment& s) -> bool {
    Walker w = walkers[warp][which];
    const bool got = w.next(a, lengths, first, S::kUnit, s);
    __syncwarp();   // every lane has read it
    if (lane == 0) walkers[warp][which] = w;
    __syncwarp();
    return got;
  };
  // ---- copies: the tiles of all segments, one after the other ----
  // Tile i of a segment holds the tokens from first_token + i kUnit on; the
  // warps' tiles of a unit follow each other.
  auto first_token = [&](const Segment& s) -> uint32_t {
    return s.span.start + s.u0 * S::kUnit + warp * S::kTile;
  };
  auto end_token = [&](const Segment& s) -> uint32_t {
    return min(s.span.end, s.span.start + s.u1 * S::kUnit);
  };
  auto tiles_of = [&](const Segment& s) -> int {
    const uint32_t from = first_token(s), stop = end_token(s);
    return from < stop ? (int)((stop - from + S::kUnit - 1) / S::kUnit) : 0;
  };
  // The next tile to copy: whether there is one, its lane's token and page
  // entry (asked for a tile ahead), and its segment's kv head and begin.
  struct Pending {
    bool more;
    uint32_t token;
    int32_t entry;
    int kv;
    uint32_t begin;
  };
  Segment source;
  int source_left = 0;          // its tiles still to copy, the next one included
  Pending next_tile = {true, 0u, -1, 0, 0u};
  auto ask = [&]() {
    while (source_left == 0) {
      if (!next_segment(1, source)) {
        next_tile.more = false;
        return;
      }
      source_left = tiles_of(source);
      next_tile.token = first_token(source) + (lane & (S::kTile - 1));
      next_tile.kv = source.kv;
      next_tile.begin = source.span.begin;
    }
    next_tile.entry = next_tile.token < end_token(source)
                          ? a.c.table[(int64_t)source.b * a.c.table_stride +
                                      (next_tile.token >> a.c.page_shift)]
                          : -1;
  };
  auto step = [&]() {   // past a tile
    if (!next_tile.more) return;
    --source_left;
    next_tile.token += S::kUnit;
    ask();
  };
  // A tile's tokens: the lane's cache row, and which tokens take part.
  struct Tokens {
    uint32_t row, here;
  };
  constexpr uint32_t kAll = S::kTile == 32 ? 0xffffffffu : 0xffffu;
  auto tokens = [&](const Pending& p) -> Tokens {
    const bool paged = p.more && (uint32_t)p.entry < (uint32_t)a.c.pages;
    Tokens k;
    k.row = paged ? (((uint32_t)p.entry * a.c.heads + p.kv) << a.c.page_shift) +
                        (p.token & ((1u << a.c.page_shift) - 1u))
                  : 0u;
    k.here = __ballot_sync(0xffffffffu, paged && p.token >= p.begin) & kAll;
    return k;
  };
  // Eight lanes copy a 128-byte line: whole lines leave L2 at once. A group of 16
  // tokens of a full tile is one run of memory when pages have at least 16;
  // otherwise every row's place comes from the lane that looked it up.
  const bool runs = a.c.page_shift >= 4;
  const int key_write = S::key_write(lane), value_write = S::value_write(lane);
  auto copy_tile = [&](const void* cache, const Tokens k, auto place) {
    if (runs && k.here == kAll) {
#pragma unroll
      for (int h = 0; h < S::kGroups; ++h) {
        const uint8_t* const src =
            static_cast<const uint8_t*>(cache) +
            (uint64_t)__shfl_sync(0xffffffffu, k.row, kGroup * h) * S::kRowBytes + lane * 16;
#pragma unroll
        for (int j = 0; j < kGroup * S::kRowBytes / 512; ++j)
          cp_async_16(place(j) + (h * (kGroup * S::kRowBytes / 512) + j) * 512, src + 512 * j);
      }
    } else {
#pragma unroll
      for (int j = 0; j < S::kKeyBytes / 512; ++j) {
        const int piece = 32 * j + lane, row = piece / (S::kRowBytes / 16);
        const uint8_t* const src =
            static_cast<const uint8_t*>(cache) +
            (uint64_t)__shfl_sync(0xffffffffu, k.row, row) * S::kRowBytes +
            piece % (S::kRowBytes / 16) * 16;
        cp_async_16(place(j) + j * 512, src, ((k.here >> row) & 1u) * 16u);
      }
    }
  };
  auto copy_keys = [&](int stage, const Tokens k) {
    const uint32_t to = stage_u32 + stage * S::kStageBytes;
    copy_tile(a.c.k, k, [&](int j) { return to + (key_write ^ S::key_write_step(j)); });
  };
  auto copy_values = [&](int stage, const Tokens k) {
    const uint32_t to = stage_u32 + S::kKeyBytes + stage * S::kStageBytes;
    copy_tile(a.c.v, k, [&](int j) { return to + (value_write ^ S::value_write_step(j)); });
  };
  // What the tokens of a tile bring to the scores: (scale of the key, log2 of
  // the value's scale a) and 1 / a, a token a lane. They are asked for with the
  // tile and put down an iteration later; with a place more than there are
  // stages, the one barrier of the warp a tile orders this too.
  // (1 for a token that takes no part: its weight is 0, whatever its slot holds)
  float key_scale = 1.f, value_scale = 1.f;
  auto ask_scales = [&](const Tokens k) {
    key_scale = value_scale = 1.f;
    if (E4M3 && ((k.here >> (lane & (S::kTile - 1))) & 1u)) {
      key_scale = a.c.k_scale[k.row >> a.c.scale_shift];
      value_scale = a.c.v_scale[k.row >> a.c.scale_shift];
    }
  };
  auto put_scales = [&](int n) {
    if (E4M3 && lane < S::kTile) {
      float* const side = side0 + (n & (S::kSides - 1)) * (3 * S::kTile);
      // a scale of 0 (nothing to add but its weight) stays finite
      const float l = log2_approx(value_scale < 0x1p-100f ? 0x1p-100f : value_scale);
      reinterpret_cast<float2*>(side)[lane] = make_float2(key_scale, l);
      side[2 * S::kTile + lane] = exp2_approx(-l);
    }
  };

  // ---- q, in the order in which the lanes hold the keys ----
  uint32_t qf[M][D / 16][4];
  float row_scale[2 * M];   // of rows g + 8 r
  auto heads_of = [&](const Segment& s, int& head0, int& rows) {
    head0 = s.kv * a.group + s.chunk * kRows;
    rows = min(kRows, (s.kv + 1) * a.group - head0);
  };
  auto ask_q = [&](const Segment& s) {
    int head0, rows;
    heads_of(s, head0, rows);
    const uint16_t* const q0 = a.q + (int64_t)s.b * a.q_stride + (int64_t)head0 * D;
#pragma unroll
    for (int step = 0; step < D / 16; ++step) {
      const int d = E4M3 ? 64 * (step >> 2) + 16 * t + 4 * (step & 3)
                         : 32 * (step >> 1) + 8 * t + 4 * (step & 1);
#pragma unroll
      for (int r = 0; r < 2 * M; ++r) {
        uint2 w = make_uint2(0u, 0u);
        if (g + 8 * r < rows) w = *reinterpret_cast<const uint2*>(q0 + (g + 8 * r) * D + d);
        qf[r >> 1][step][r & 1] = w.x;
        qf[r >> 1][step][2 + (r & 1)] = w.y;
      }
    }
  };
  auto convert_q = [&]() {
#pragma unroll
    for (int r = 0; r < 2 * M; ++r) row_scale[r] = a.scale * 1.4426950408889634f;
    if (E4M3) {
#pragma unroll
      for (int r = 0; r < 2 * M; ++r) {
        float top = 0.f;
#pragma unroll
        for (int step = 0; step < D / 16; ++step)
#pragma unroll
          for (int i = r & 1; i < 4; i += 2)
            top = fmaxf(top, fmaxf(fabsf(bf16_lo(qf[r >> 1][step][i])),
                                   fabsf(bf16_hi(qf[r >> 1][step][i]))));
        top = quad_max(top);
        // a power of two brings the head's largest element into [1, 2)
        const uint32_t e = min(max((__float_as_uint(top) >> 23) & 255u, 1u), 253u);
        const float down = __uint_as_float((254u - e) << 23);
        row_scale[r] *= __uint_as_float(e << 23);
#pragma unroll
        for (int step = 0; step < D / 16; ++step)
#pragma unroll
          for (int i = r & 1; i < 4; i += 2) {
            uint32_t& w = qf[r >> 1][step][i];
            w = pack_f16(bf16_lo(w) * down, bf16_hi(w) * down);
          }
      }
    }
  };

  // ---- the first tiles and the first q, all asked for before any is used ----
  // The keys of a tile are one group of copies and its values the next, so
  // that a stage's keys make room for a later tile's while its values are
  // still to be used. Every wait leaves all but the group it needs pending.
  uint32_t here[S::kStages];   // of the next tiles
  Pending firsts[S::kStages];
  ask();
#pragma unroll
  for (int i = 0; i < S::kStages; ++i) {
    firsts[i] = next_tile;
    step();
  }
  Segment seg;
  const int key_read = S::key_read(g, t), value_read = S::value_read(g, t);
  int stage = 0, n = 0;   // of the next tile: its stage, and its number (for put_scales)
  bool running = next_segment(0, seg);
  if (running && !S::kSharedQ) ask_q(seg);
  {
    float ks[S::kStages], vs[S::kStages];
#pragma unroll
    for (int i = 0; i < S::kStages; ++i) {
      const Tokens k = tokens(firsts[i]);
      here[i] = k.here;
      if (firsts[i].more) copy_keys(i, k);
      cp_commit();
      if (firsts[i].more) copy_values(i, k);
      cp_commit();
      ask_scales(k);
      ks[i] = key_scale;
      vs[i] = value_scale;
    }
#pragma unroll
    for (int i = 0; i < S::kStages; ++i) {
      key_scale = ks[i];
      value_scale = vs[i];
      if (i + 1 < S::kStages) put_scales(i);
    }
  }
  uint4* const shared_q =
      reinterpret_cast<uint4*>(smem + kWarps * S::kWarpBytes + 2 * S::kJoinBytes) + lane;
  while (running) {
    if (S::kSharedQ) ask_q(seg);
    convert_q();
    if (S::kSharedQ) {   // (all warps have left the last segment's tiles)
#pragma unroll
      for (int step = 0; step < D / 16; ++step)
        if (step % kWarps == warp) {
#pragma unroll
          for (int m = 0; m < M; ++m)
            shared_q[32 * (M * step + m)] = make_uint4(qf[m][step][0], qf[m][step][1],
                                                       qf[m][step][2], qf[m][step][3]);
        }
      __syncthreads();
    }
    const int tiles = tiles_of(seg);

    // q's operands of contraction step `step`
    auto q_of = [&](int m, int step, uint32_t (&q)[4]) {
      uint4 v = make_uint4(qf[m][step][0], qf[m][step][1], qf[m][step][2], qf[m][step][3]);
      if (S::kSharedQ) v = shared_q[32 * (M * step + m)];
      q[0] = v.x;
      q[1] = v.y;
      q[2] = v.z;
      q[3] = v.w;
    };

    float acc[M][D / 8][4];
    float top[2 * M], sum[2 * M];   // of rows g + 8 r
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[m][i][j] = 0.f;
#pragma unroll
    for (int r = 0; r < 2 * M; ++r) {
      top[r] = -INFINITY;
      sum[r] = 0.f;
    }

    for (int i = 0; i < tiles; ++i, ++n) {
      const uint8_t* const tile = stage0 + stage * S::kStageBytes;
      const float* const side = side0 + (n & (S::kSides - 1)) * (3 * S::kTile);
      put_scales(n + S::kStages - 1);
      cp_wait<2 * S::kStages - 1>();   // this tile's keys
      __syncwarp();

      // scores: [heads g + 8 r] x [tokens 8 n + 2 t, + 1]
      float x[M][2 * S::kGroups][4];
#pragma unroll
      for (int h = 0; h < S::kGroups; ++h) {
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) x[m][2 * h + n][j] = 0.f;
#pragma unroll
        for (int p = 0; p < S::kKeyPieces; ++p) {
          uint4 w[2];
#pragma unroll
          for (int n = 0; n < 2; ++n)
            w[n] = *reinterpret_cast<const uint4*>(
                tile + (key_read ^ ((p & 1) * 64)) + 128 * (p >> 1) +
                8 * (2 * h + n) * S::kRowBytes);
          if (E4M3) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t b[2][2];
#pragma unroll
              for (int n = 0; n < 2; ++n)
                e4m3x4_to_f16(j == 0 ? w[n].x : j == 1 ? w[n].y : j == 2 ? w[n].z : w[n].w,
                              b[n][0], b[n][1]);
#pragma unroll
              for (int m = 0; m < M; ++m) {
                uint32_t aq[4];
                q_of(m, 4 * p + j, aq);
#pragma unroll
                for (int n = 0; n < 2; ++n)
                  mma16816<true>(x[m][2 * h + n], aq, b[n][0], b[n][1]);
              }
            }
          } else {
#pragma unroll
            for (int m = 0; m < M; ++m) {
              uint32_t a0[4], a1[4];
              q_of(m, 2 * p, a0);
              q_of(m, 2 * p + 1, a1);
#pragma unroll
              for (int n = 0; n < 2; ++n) {
                mma16816<false>(x[m][2 * h + n], a0, w[n].x, w[n].y);
                mma16816<false>(x[m][2 * h + n], a1, w[n].z, w[n].w);
              }
            }
          }
        }
        // base 2, with the value rows' scales in the exponent
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          float4 sc = make_float4(1.f, 0.f, 1.f, 0.f);
          if (E4M3)
            sc = *reinterpret_cast<const float4*>(side + 2 * (8 * (2 * h + n) + 2 * t));
#pragma unroll
          for (int r = 0; r < 2 * M; ++r) {
            float* const y = x[r >> 1][2 * h + n] + 2 * (r & 1);
            if (E4M3) {
              y[0] = fmaf(y[0] * sc.x, row_scale[r], sc.y);
              y[1] = fmaf(y[1] * sc.z, row_scale[r], sc.w);
            } else {
              y[0] *= row_scale[r];
              y[1] *= row_scale[r];
            }
          }
        }
      }
      // the tile after the stages' takes the place of these keys
      __syncwarp();
      const bool copies = next_tile.more;
      const Tokens next = tokens(next_tile);
      if (copies) copy_keys(stage, next);
      cp_commit();

      if (here[0] != kAll) {
#pragma unroll
        for (int n = 0; n < 2 * S::kGroups; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (!((here[0] >> (8 * n + 2 * t + (j & 1))) & 1u)) {
#pragma unroll
              for (int m = 0; m < M; ++m) x[m][n][j] = -INFINITY;
            }
      }
#pragma unroll
      for (int j = 0; j + 1 < S::kStages; ++j) {
        here[j] = here[j + 1];
      }
      here[S::kStages - 1] = next.here;
      ask_scales(next);
      step();

      // a tile that passes the bound moves it
      float high[2 * M];
      bool moves = false;
#pragma unroll
      for (int r = 0; r < 2 * M; ++r) {
        const float* const y0 = x[r >> 1][0] + 2 * (r & 1);
        high[r] = fmaxf(y0[0], y0[1]);
#pragma unroll
        for (int n = 1; n < 2 * S::kGroups; ++n) {
          const float* const y = x[r >> 1][n] + 2 * (r & 1);
          high[r] = fmaxf(high[r], fmaxf(y[0], y[1]));
        }
        moves = moves || high[r] > top[r] + kMostWeight;
      }
      if (__any_sync(0xffffffffu, moves)) {
#pragma unroll
        for (int r = 0; r < 2 * M; ++r) {
          const float was = top[r];
          top[r] = fmaxf(was, quad_max(high[r]) - kNewWeight);
          const float f = weight(was, top[r]);
          sum[r] *= f;
#pragma unroll
          for (int n = 0; n < D / 8; ++n) {
            acc[r >> 1][n][2 * (r & 1)] *= f;
            acc[r >> 1][n][2 * (r & 1) + 1] *= f;
          }
        }
      }
      // weights
      uint32_t wf[M][S::kGroups][4], wr[M][S::kGroups][4];
#pragma unroll
      for (int n = 0; n < 2 * S::kGroups; ++n) {
        float2 inverse = make_float2(1.f, 1.f);
        if (E4M3)
          inverse = *reinterpret_cast<const float2*>(side + 2 * S::kTile + 8 * n + 2 * t);
#pragma unroll
        for (int r = 0; r < 2 * M; ++r) {
          const float bound = top[r] == -INFINITY ? 0.f : top[r];
          const float* const y = x[r >> 1][n] + 2 * (r & 1);
          const float w0 = exp2_approx(y[0] - bound), w1 = exp2_approx(y[1] - bound);
          const int e = 2 * (n & 1) + (r & 1);
          uint32_t& to = wf[r >> 1][n >> 1][e];
          if (E4M3) {
            sum[r] = fmaf(w0, inverse.x, fmaf(w1, inverse.y, sum[r]));
            to = pack_f16(w0, w1);
          } else {
            sum[r] += w0 + w1;
            to = pack_bf16(w0, w1);
            wr[r >> 1][n >> 1][e] = pack_bf16(w0 - bf16_lo(to), w1 - bf16_hi(to));
          }
        }
      }
      cp_wait<2 * S::kStages - 1>();   // this tile's values
      __syncwarp();
      // acc += weights x values, tile (p, j): element j of the lanes' pieces p
      const uint8_t* const values = tile + S::kKeyBytes;
#pragma unroll
      for (int h = 0; h < S::kGroups; ++h)
#pragma unroll
        for (int p = 0; p < S::kValuePieces; ++p) {
          uint32_t w[4][S::kPieceBytes / 4];
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            const int r = 8 * (n >> 1) + (n & 1);
            const uint8_t* const piece =
                S::kRowBytes == 64
                    ? values + (value_read ^ ((n & 1) * 64)) + (kGroup * h + (r & 8)) * S::kRowBytes
                    : values + value_read + (kGroup * h + r) * S::kRowBytes + 128 * p;
            if (S::kPieceBytes == 16) {
              const uint4 raw = *reinterpret_cast<const uint4*>(piece);
              w[n][0] = raw.x;
              w[n][1] = raw.y;
              w[n][S::kPieceBytes / 4 - 2] = raw.z;
              w[n][S::kPieceBytes / 4 - 1] = raw.w;
            } else {
              const uint2 raw = *reinterpret_cast<const uint2*>(piece);
              w[n][0] = raw.x;
              w[n][1] = raw.y;
            }
          }
#pragma unroll
          for (int j = 0; j < S::kPieceBytes / 4; ++j) {
            if (E4M3) {
              // bytes 4j .. 4j+3 of tokens (2t, 2t+1) and (2t+8, 2t+9), paired
              uint32_t b[4][2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                e4m3x4_to_f16(__byte_perm(w[2 * e][j], w[2 * e + 1][j], 0x5140), b[0][e],
                              b[1][e]);
                e4m3x4_to_f16(__byte_perm(w[2 * e][j], w[2 * e + 1][j], 0x7362), b[2][e],
                              b[3][e]);
              }
#pragma unroll
              for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int m = 0; m < M; ++m)
                  mma16816<true>(acc[m][p * S::kChunk + 4 * j + k], wf[m][h], b[k][0], b[k][1]);
            } else {
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const uint32_t pick = k == 0 ? 0x5410 : 0x7632;
                const uint32_t b0 = __byte_perm(w[0][j], w[1][j], pick);
                const uint32_t b1 = __byte_perm(w[2][j], w[3][j], pick);
#pragma unroll
                for (int m = 0; m < M; ++m) {
                  mma16816<false>(acc[m][p * S::kChunk + 2 * j + k], wf[m][h], b0, b1);
                  mma16816<false>(acc[m][p * S::kChunk + 2 * j + k], wr[m][h], b0, b1);
                }
              }
            }
          }
        }
      __syncwarp();
      if (copies) copy_values(stage, next);
      cp_commit();
      stage = stage + 1 == S::kStages ? 0 : stage + 1;
    }

    // ---- join the warps ----
    const Segment done = seg;
    running = next_segment(0, seg);
    if (running && !S::kSharedQ) ask_q(seg);
#pragma unroll
    for (int r = 0; r < 2 * M; ++r) sum[r] = quad_sum(sum[r]);
    auto put_acc = [&](int to) {
      if (t == 0) {
#pragma unroll
        for (int r = 0; r < 2 * M; ++r) stats[to][g + 8 * r] = make_float2(top[r], sum[r]);
      }
#pragma unroll
      for (int r = 0; r < 2 * M; ++r) {
        float4* const row = reinterpret_cast<float4*>(join0 + to * S::kJoinBytes) +
                            (g + 8 * r) * (D / 4);
#pragma unroll
        for (int p = 0; p < S::kValuePieces; ++p)
#pragma unroll
          for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int j = 0; j < S::kChunk / 4; ++j) {
              const int i = p * S::kChunk + 4 * j, e = 2 * (r & 1) + half;
              const int f = ((p * 8 + 2 * t + half) * S::kChunk) / 4 + j;
              const float (&from)[D / 8][4] = acc[r >> 1];
              row[join_place<S::kChunk>(g, f)] =
                  make_float4(from[i][e], from[i + 1][e], from[i + 2][e], from[i + 3][e]);
            }
      }
    };
    __syncthreads();   // the last segment's has been read
    if (warp >= 2) put_acc(warp - 2);
    __syncthreads();
    if (warp < 2) {
#pragma unroll
      for (int r = 0; r < 2 * M; ++r) {
        const float2 other = stats[warp][g + 8 * r];
        const float m = fmaxf(top[r], other.x);
        const float mine = weight(top[r], m), its = weight(other.x, m);
        top[r] = m;
        sum[r] = sum[r] * mine + other.y * its;
        const float4* const row = reinterpret_cast<const float4*>(join0 + warp * S::kJoinBytes) +
                                  (g + 8 * r) * (D / 4);
#pragma unroll
        for (int p = 0; p < S::kValuePieces; ++p)
#pragma unroll
          for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int j = 0; j < S::kChunk / 4; ++j) {
              const int i = p * S::kChunk + 4 * j, e = 2 * (r & 1) + half;
              const int f = ((p * 8 + 2 * t + half) * S::kChunk) / 4 + j;
              float (&to)[D / 8][4] = acc[r >> 1];
              const float4 v = row[join_place<S::kChunk>(g, f)];
              to[i][e] = to[i][e] * mine + v.x * its;
              to[i + 1][e] = to[i + 1][e] * mine + v.y * its;
              to[i + 2][e] = to[i + 2][e] * mine + v.z * its;
              to[i + 3][e] = to[i + 3][e] * mine + v.w * its;
            }
      }
      __syncwarp();   // every lane has read the statistics it replaces
      put_acc(warp);
    }
    __syncthreads();
    int head0, rows;
    heads_of(done, head0, rows);
    const bool whole = done.whole();
    const int64_t slot = 2 * worker + (done.u0 == 0 ? 1u : 0u);
    for (int i = threadIdx.x; i < rows * (D / 4); i += kThreads) {
      const int row = i / (D / 4), f = i % (D / 4);
      const float2 s0 = stats[0][row], s1 = stats[1][row];
      const float m = fmaxf(s0.x, s1.x);
      const float k0 = weight(s0.x, m), k1 = weight(s1.x, m);
      const int at = row * (D / 4) + join_place<S::kChunk>(row, f);
      const float4 v0 = reinterpret_cast<const float4*>(join0)[at];
      const float4 v1 = reinterpret_cast<const float4*>(join0 + S::kJoinBytes)[at];
      const float l = s0.y * k0 + s1.y * k1;
      const float4 o = make_float4(v0.x * k0 + v1.x * k1, v0.y * k0 + v1.y * k1,
                                   v0.z * k0 + v1.z * k1, v0.w * k0 + v1.w * k1);
      if (whole) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int64_t to = (int64_t)done.b * a.q_heads + head0 + row;
        *reinterpret_cast<uint2*>(a.out + to * D + 4 * f) =
            make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
        if (f == 0 && a.lse != nullptr) a.lse[to] = (m + log2f(l)) * 0.6931471805599453f;
      } else {
        reinterpret_cast<float4*>(a.parts)[(slot * kRows + row) * (D / 4) + f] = o;
        if (f == 0) a.stats[slot * kRows + row] = make_float2(m, l);
      }
    }
    if (done.u0 == 0 && threadIdx.x == 0 && !a.whole) {
      Joint j;
      j.item = (int32_t)(((int64_t)done.b * a.c.heads + done.kv) * a.chunks + done.chunk);
      j.first = (int32_t)worker;
      j.pieces = 1;
      j.pad = 0;
      if (!whole) {
        // place p belongs to the largest worker w with floor(total w / workers) <= p
        const uint32_t last = min(
            (uint32_t)(((uint64_t)done.end * workers + total - 1) / total), workers) - 1;
        j.pieces = (int32_t)(last - worker + 1);
      }
      if (!a.by_worker) a.joints[j.item] = j;
      else if (!whole) a.joints[worker] = j;   // (a worker has one such item at most)
    }
  }
  cp_wait<0>();   // (only empty groups are left)
}

// Joins the pieces of the items that several workers share. A block takes one
// item's rows, or a share of them when there are few items; a row gets `share` warps (a
// power of two), each of which takes every so many-th piece with a running bound.
constexpr int kJoinWarps = 16;

template <int D, int M>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const Args a, int unit,
                                                                int share) {
  constexpr int kRows = M * kMmaRows;
  constexpr int N = D / 32;
  __shared__ float2 stats[kJoinWarps];
  __shared__ float sacc[kJoinWarps][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int items = a.c.heads * a.chunks;
  const int row = blockIdx.y * (kJoinWarps / share) + warp / share;
  // by item, one of a context without tokens has no joint
  const bool none =
      !a.by_worker && span_of(a, a.lengths[blockIdx.x / items], unit).units == 0;
  pdl_wait();
  if (none) return;
  const Joint j = a.joints[blockIdx.x];
  // (lengths that changed under the kernels can leave an item's joint unwritten: what
  // the workspace held must not lead out of it or of the outputs)
  if (j.pieces < 2 || (uint32_t)j.item >= (uint32_t)(a.batch * items) || j.first < 0 ||
      j.first > kMaxWorkers - j.pieces)
    return;
  const int b = j.item / items, item = j.item - b * items;
  const int kv = item / a.chunks;
  const int head0 = kv * a.group + (item - kv * a.chunks) * kRows;
  const int rows = min(kRows, (kv + 1) * a.group - head0);
  float m = -INFINITY, l = 0.f, acc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = 0.f;
  if (row < rows) {
    constexpr int kBatch = 8;   // pieces asked for together
    for (int p0 = warp & (share - 1); p0 < j.pieces; p0 += kBatch * share) {
      float2 st[kBatch];
      float v[kBatch][N];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int p = p0 + k * share;
        st[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int i = 0; i < N; ++i) v[k][i] = 0.f;
        if (p >= j.pieces) continue;
        const int64_t slot = 2 * (int64_t)(j.first + p) + (p == 0 ? 1 : 0);
        st[k] = a.stats[slot * kRows + row];
        const float* from = a.parts + (slot * kRows + row) * D + lane * N;
#pragma unroll
        for (int i = 0; i < N; i += 2)
          *reinterpret_cast<float2*>(v[k] + i) = *reinterpret_cast<const float2*>(from + i);
      }
      float top = m;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) top = fmaxf(top, st[k].x);
      const float was = weight(m, top);
      m = top;
      l *= was;
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] *= was;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const float w = weight(st[k].x, m);
        l = fmaf(st[k].y, w, l);
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] = fmaf(v[k][i], w, acc[i]);
      }
    }
  }
  if (share > 1) {   // join the row's warps, in its first one
    if (lane == 0) stats[warp] = make_float2(m, l);
#pragma unroll
    for (int i = 0; i < N; ++i) sacc[warp][i * 32 + lane] = acc[i];
    __syncthreads();
    if ((warp & (share - 1)) != 0) return;
    for (int w = warp; w < warp + share; ++w) m = fmaxf(m, stats[w].x);
    l = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.f;
    for (int w = warp; w < warp + share; ++w) {
      const float k = weight(stats[w].x, m);
      l = fmaf(stats[w].y, k, l);
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] = fmaf(sacc[w][i * 32 + lane], k, acc[i]);
    }
  }
  if (row >= rows) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int64_t at = (int64_t)b * a.q_heads + head0 + row;
#pragma unroll
  for (int i = 0; i < N; i += 2)
    *reinterpret_cast<uint32_t*>(a.out + at * D + lane * N + i) =
        pack_bf16(acc[i] * inv, acc[i + 1] * inv);
  if (lane == 0 && a.lse != nullptr) a.lse[at] = (m + log2f(l)) * 0.6931471805599453f;
}

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

// Whether items can have two tensor core tiles of query heads, and whether they do:
// two tiles save half the copies and conversions of a token and put down twice as much
// an item. Measured with 20 heads a kv head (one tile, two tiles): 2^17 tokens of 128 e4m3
// elements 22.8, 24.8 us; 2^18 33.0, 32.5; 2^19 51.1, 46.4; of 128 bf16 elements 25.9,
// 28.3; 39.2, 39.7; 83.3, 60.6; of 64 e4m3 15.4, 16.3; 21.4, 21.2; 33.0, 30.7. The
// lengths are on the device: the table's room stands for them.
bool two_tiles_fit(int group, int head_dim) { return group > kMmaRows && head_dim <= 128; }
constexpr int64_t kTwoTileTokens = 1 << 18;
int chunks_of(int group, int rows) { return (group + rows - 1) / rows; }

int64_t table_room(const CacheView& c) {
  return std::min<int64_t>((int64_t)c.max_pages << c.page_shift, 0x7fffffff);
}

template <bool E4M3, int D, int M>
int launch(const Args& a, cudaStream_t stream) {
  using S = Shape<E4M3, D, M>;
  const int64_t items = (int64_t)a.batch * a.c.heads * a.chunks;
  const int64_t room = table_room(a.c);
  // units of the longest context the table can hold (a window's can start
  // before it by a group)
  const int64_t units = (room + kGroup + S::kUnit - 1) / S::kUnit;
  if (items * (units + kItemCost) >= (int64_t(1) << 31)) return -2;
  // the opt-in to more than 48 KB of shared memory, once per device
  static std::atomic<uint64_t> opted{0};
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess) return -3;
  const uint64_t bit = uint64_t(1) << (device & 63);
  if ((opted.load(std::memory_order_relaxed) & bit) == 0 || device >= 64) {
    if (cudaFuncSetAttribute(paged_attention_kernel<E4M3, D, M>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             S::kSmemBytes) != cudaSuccess)
      return -3;
    opted.fetch_or(bit, std::memory_order_relaxed);
  }
  Args args = a;
  args.whole = room <= kWholeUnits * S::kUnit && items <= kSms * S::kCtas;
  const int grid = (int)std::min<int64_t>(kSms * S::kCtas,
                                          args.whole ? items : items * (units + kItemCost));
  args.joint_count = (int)std::min<int64_t>(items, grid);
  args.by_worker = args.joint_count < items;
  cudaError_t e = launch_kernel(true, dim3(grid), dim3(kThreads), S::kSmemBytes, stream,
                                paged_attention_kernel<E4M3, D, M>, args);
  if (e != cudaSuccess) return -3;
  if (args.whole) return 0;
  // few items: a row's pieces go to several warps (2 blocks an SM hold 16 each)
  int share = 1;
  while (share < kJoinWarps && 2 * share * args.joint_count <= 2 * kSms) share *= 2;
  e = launch_kernel(true, dim3(args.joint_count, share * M), dim3(kJoinWarps * 32), 0, stream,
                    join_kernel<D, M>, args, S::kUnit, share);
  return e == cudaSuccess ? 0 : -3;
}

// The workspace's parts: the joints, at most one a worker, then the slots' statistics
// and rows. The size does not depend on the batch, so that a buffer serves every batch.
struct Parts {
  size_t joints, stats, rows;
};
Parts parts_of(int group, int head_dim) {
  const size_t slot_rows =
      (size_t)2 * kMaxWorkers * (two_tiles_fit(group, head_dim) ? 2 : 1) * kMmaRows;
  return {align256(kMaxWorkers * sizeof(Joint)), align256(slot_rows * sizeof(float2)),
          slot_rows * head_dim * sizeof(float)};
}

}  // namespace

size_t paged_attention_ws_bytes(int heads, int head_dim, int q_heads) {
  const Parts p = parts_of(q_heads / heads, head_dim);
  return p.joints + p.stats + p.rows;
}

int launch_paged_attention(const CacheView& c, const uint16_t* q, int64_t q_stride, int batch,
                           int q_heads, const int32_t* lengths, float scale, int window,
                           uint16_t* out, float* lse, void* ws, cudaStream_t stream) {
  Args a{};
  a.c = c;
  a.q = q;
  a.q_stride = q_stride;
  a.batch = batch;
  a.q_heads = q_heads;
  a.group = q_heads / c.heads;
  const int64_t reach = window > 0 ? std::min<int64_t>(window, table_room(c)) : table_room(c);
  const int64_t spans = (int64_t)batch * c.heads;
  const bool two = two_tiles_fit(a.group, c.head_dim) &&
                   reach >= (kTwoTileTokens + spans - 1) / spans;
  a.rows = (two ? 2 : 1) * kMmaRows;
  a.chunks = chunks_of(a.group, a.rows);
  a.lengths = lengths;
  a.scale = scale;
  a.window = window;
  a.out = out;
  a.lse = lse;
  const Parts parts = parts_of(a.group, c.head_dim);
  uint8_t* const p = static_cast<uint8_t*>(ws);
  a.joints = reinterpret_cast<Joint*>(p);
  a.stats = reinterpret_cast<float2*>(p + parts.joints);
  a.parts = reinterpret_cast<float*>(p + parts.joints + parts.stats);
  if (c.e4m3) {
    if (c.head_dim == 64)
      return two ? launch<true, 64, 2>(a, stream) : launch<true, 64, 1>(a, stream);
    if (c.head_dim == 128)
      return two ? launch<true, 128, 2>(a, stream) : launch<true, 128, 1>(a, stream);
    return launch<true, 256, 1>(a, stream);
  }
  if (c.head_dim == 64)
    return two ? launch<false, 64, 2>(a, stream) : launch<false, 64, 1>(a, stream);
  if (c.head_dim == 128)
    return two ? launch<false, 128, 2>(a, stream) : launch<false, 128, 1>(a, stream);
  return launch<false, 256, 1>(a, stream);
}

}  // namespace moe
