// The key-value cache's write where a page has one scale for each head, behind the
// rotation of the keys when there is one.
//
//   a = max |x| over the tokens that the call brings to the page,
//   s(a) = 2^e, e the least integer >= -48 with a <= 448 * 2^e,
//   scale' = s(a) when the call begins the page (writes its offset 0),
//            max(scale, s(a)) when not; then a code q that stays becomes
//            e4m3(q scale / scale'), and x is stored as e4m3(x / scale').
//
// Scales are powers of two, so that quotients by them are exact and a code has one
// rounding; a code that stays is exact under a grown scale as long as it is not
// subnormal there. e4m3 spans 2^-9 to 448, so that against a scale that brings the
// largest element to 448 a power of two costs at most the lowest binade of those 18.
//
// A team of one or four warps takes the runs of tokens that begin in its part of the call,
// for one head of k or v. A run is what the call brings to one page: tokens that follow
// one another with slots of the same page. Its maximum has to be known before its first
// code, so the first 4 units of a thread stay in registers between, and the rest are read
// twice: one warp for pages of up to 16 tokens of 128 elements, four for larger ones. Bound by
// memory without a rotation: 2 bytes an element in, 1 out; GB300, 12100 tokens of 8 heads of
// 128 in pages of 16: 21 us, 3.5 TB/s of the copy's 6.8 (with fp32 elements kept instead of what
// was read, 16 warps an SM and 42 us). Behind a rotation by the angles: a block works a run's
// out once for up to four of k's heads. q is rotated by a launch of its own (28 us with 64
// heads and 6146 tokens), which runs beside this one's last blocks: 49 us together with 4
// heads of k and v (59 one after the other; 53 with the angles worked out for each head).
#include <algorithm>

#include "attention.h"
#include "common.cuh"
#include "internal.h"
#include "rotary.cuh"

#include <cuda_fp16.h>

namespace moe {

namespace {

constexpr int kWarps = 4;       // of a block
constexpr int kKept = 4;        // units of a thread in registers
constexpr int kMostTokens = 64; // of a team's part
constexpr int kMostHeads = 4;   // of k that a team does one after the other
constexpr int kTurns = 4096;    // (cos, sin) of a block
constexpr float kLeastScale = 0x1p-48f;

// 2^e, e the least integer >= -48 with amax <= 448 * 2^e (448 = 1.75 * 2^8).
__device__ __forceinline__ float page_scale(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const int e = (int)(bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return fmaxf(__uint_as_float((uint32_t)max(e, 1) << 23), kLeastScale);
}

__device__ __forceinline__ uint2 codes8(const float* v, float by) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    w[i] = (uint32_t)f32x2_to_e4m3x2(v[4 * i] * by, v[4 * i + 1] * by) |
           ((uint32_t)f32x2_to_e4m3x2(v[4 * i + 2] * by, v[4 * i + 3] * by) << 16);
  return make_uint2(w[0], w[1]);
}

// Four codes times a power of two, as codes.
__device__ __forceinline__ uint32_t scaled_codes(uint32_t w, float by) {
  uint32_t out = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(w >> (16 * i))));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    out |= (uint32_t)f32x2_to_e4m3x2(f.x * by, f.y * by) << (16 * i);
  }
  return out;
}

// TEAM: warps of a team.
template <int PAIRS, int TEAM>
__global__ void __launch_bounds__(32 * kWarps, PAIRS == kNoPairs ? 8 : 4)
    page_write_kernel(const RotaryArgs a, int part, int at_once) {
  constexpr int kThreads = 32 * TEAM, kMine = kTurns / (kWarps / TEAM);
  // (cos, sin) of a run's tokens, for all of the team's heads
  __shared__ __align__(16) float2 all_turns[PAIRS == kNoPairs ? 1 : kTurns];
  // of each team: the slots of its part and of the token before it; its warps' findings
  __shared__ int32_t all_slots[kWarps / TEAM][kMostTokens + 1];
  __shared__ int ends[TEAM], begins[TEAM];
  __shared__ float maxima[2][TEAM];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, team = threadIdx.x / kThreads, me = threadIdx.x % kThreads;
  const int warp = me >> 5;
  const int64_t t_begin = ((int64_t)blockIdx.x * (kWarps / TEAM) + team) * part;
  if (TEAM == 1 && t_begin >= a.T) return;
  const int t0 = (int)t_begin, here = min(part, a.T - t0);
  // k's heads in groups, then v's
  const int groups = PAIRS == kNoPairs ? a.k_heads : (a.k_heads + at_once - 1) / at_once;
  const bool is_v = (int)blockIdx.y >= groups;
  const int head0 = is_v ? (int)blockIdx.y - groups
                         : (int)blockIdx.y * (PAIRS == kNoPairs ? 1 : at_once);
  const int head1 = PAIRS == kNoPairs || is_v ? head0 + 1 : min(a.k_heads, head0 + at_once);
  float2* const turns = all_turns + (PAIRS == kNoPairs ? 0 : team * kMine);
  const int size = 1 << a.page_shift;
  int32_t* const slots = all_slots[team];
  auto sync = [&]() {
    if (TEAM == 1) __syncwarp(); else __syncthreads();
  };
  for (int i = me; i <= here; i += kThreads) slots[i] = t0 + i > 0 ? a.slots[t0 + i - 1] : -1;
  sync();
  // the page of a slot (-1: none)
  auto page_of = [&](int32_t slot) -> int {
    return (uint32_t)slot < a.cache_slots ? slot >> a.page_shift : -1;
  };

  const int units = a.head_dim / kUnit, u = me % units;   // of a token
  const int first = me / units, step = kThreads / units;  // tokens
  const int rot_units = PAIRS == kNoPairs || is_v ? 0 : a.rot / kUnit;
  const bool rotates = u < rot_units;
  const int from = rotates || rot_units == 0 ? 0 : a.rot;
  const int region = rot_units == 0 ? a.head_dim : rotates ? a.rot : a.head_dim - a.rot;
  const int run0 = from + 8 * (rotates ? u : u - rot_units), run1 = run0 + region / 2;
  const int64_t stride = is_v ? a.v_stride : a.k_stride;
  // a unit as it comes, and its elements (rotated)
  struct Raw {
    uint4 a, b;
  };
  const uint16_t* src = (is_v ? a.v : a.k) + head0 * a.head_dim;   // of the head
  auto ask = [&](int t) -> Raw {
    return {*reinterpret_cast<const uint4*>(src + t * stride + run0),
            *reinterpret_cast<const uint4*>(src + t * stride + run1)};
  };
  const int pairs = a.rot / 2, room = PAIRS == kNoPairs ? 0 : kMine / pairs;   // tokens
  auto elements = [&](const Raw& raw, int t, int in_run, float* x) {
    unpack8(raw.a, x);
    unpack8(raw.b, x + 8);
    if (PAIRS != kNoPairs && rotates) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int p = pair_of<PAIRS>(u, j, a.rot);
        const float2 cs = in_run < room ? turns[in_run * pairs + p]
                                        : turn_of(a, t, a.turns[p], a.pair_axis[p]);
        turn_pair(cs, PAIRS == kNeighbours ? x[2 * j] : x[j],
                  PAIRS == kNeighbours ? x[2 * j + 1] : x[8 + j]);
      }
    }
  };
  auto largest = [&](const float* x) {
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < kUnit; ++j) m = fmaxf(m, fabsf(x[j]));
    return m;
  };

  for (int i = 0; i < here; ++i) {
    const int page = page_of(slots[i + 1]);
    if (page < 0 || page == page_of(slots[i])) continue;
    // the run: tokens [t, t + n), and whether it begins the page
    const int t = t0 + i;
    int end = size, zero = size;   // (slots differ, so that a run has at most `size` tokens)
    for (int j = me; j < size; j += kThreads) {
      const int32_t slot = t + j < a.T ? a.slots[t + j] : -1;
      if (page_of(slot) != page) {
        end = j;
        break;
      }
      if ((slot & (size - 1)) == 0) zero = min(zero, j);
    }
    end = __reduce_min_sync(0xffffffffu, end);
    zero = __reduce_min_sync(0xffffffffu, zero);
    if (TEAM > 1) {
      if (lane == 0) {
        ends[warp] = end;
        begins[warp] = zero;
      }
      __syncthreads();
#pragma unroll
      for (int w = 0; w < TEAM; ++w) {
        end = min(end, ends[w]);
        zero = min(zero, begins[w]);
      }
    }
    const int n = end;
    const bool begun = zero < n;
    if (PAIRS != kNoPairs && !is_v) {
      sync();   // (the last run's have been used)
      for (int c = me; c < min(n, room) * pairs; c += kThreads) {
        const int j = c / pairs, p = c - j * pairs;
        turns[c] = turn_of(a, t + j, a.turns[p], a.pair_axis[p]);
      }
      sync();
    }
    for (int head = head0; head < (PAIRS == kNoPairs ? head0 + 1 : head1); ++head) {
      if (PAIRS != kNoPairs) src = (is_v ? a.v : a.k) + head * a.head_dim;
      const int64_t block = (int64_t)page * a.k_heads + head;
      float* const scale_at = (is_v ? a.v_scale : a.k_scale) + block;
      const float was = begun ? 0.f : *scale_at;

      // (rotated units are kept as they are wanted, others as they come)
      Raw raw[PAIRS == kNoPairs ? kKept : 1];
      float x[PAIRS == kNoPairs ? 1 : kKept][kUnit], top = 0.f;
      if (PAIRS == kNoPairs) {
#pragma unroll
        for (int k = 0; k < kKept; ++k)
          if (first + k * step < n) raw[PAIRS == kNoPairs ? k : 0] = ask(t + first + k * step);
      }
#pragma unroll
      for (int k = 0; k < kKept; ++k) {
        const int j = first + k * step;
        if (j < n) {
          float* const y = x[PAIRS == kNoPairs ? 0 : k];
          elements(PAIRS == kNoPairs ? raw[PAIRS == kNoPairs ? k : 0] : ask(t + j), t + j, j, y);
          top = fmaxf(top, largest(y));
        }
      }
      for (int j = first + kKept * step; j < n; j += step) {
        float y[kUnit];
        elements(ask(t + j), t + j, j, y);
        top = fmaxf(top, largest(y));
      }
      top = warp_max(top);
      if (TEAM > 1) {
        float(&of)[TEAM] = maxima[head & 1];   // (the next head's can come before all have read)
        if (lane == 0) of[warp] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < TEAM; ++w) top = fmaxf(top, of[w]);
      }
      const float scale = fmaxf(was, page_scale(top)), by = __frcp_rn(scale);
      uint8_t* const out = static_cast<uint8_t*>(is_v ? a.cache_v : a.cache_k) +
                           (block << a.page_shift) * a.head_dim;
      if (!begun && scale > was) {   // the codes that stay (the run's are written over them)
        const float down = was * by;
        for (int c = me; c < size * a.head_dim / 16; c += kThreads) {
          uint4 w = reinterpret_cast<uint4*>(out)[c];
          w.x = scaled_codes(w.x, down);
          w.y = scaled_codes(w.y, down);
          w.z = scaled_codes(w.z, down);
          w.w = scaled_codes(w.w, down);
          reinterpret_cast<uint4*>(out)[c] = w;
        }
        sync();
      }
      auto store = [&](int t, const float* x) {
        uint8_t* const row = out + (a.slots[t] & (size - 1)) * a.head_dim;
        *reinterpret_cast<uint2*>(row + run0) = codes8(x, by);
        *reinterpret_cast<uint2*>(row + run1) = codes8(x + 8, by);
      };
#pragma unroll
      for (int k = 0; k < kKept; ++k) {
        const int j = first + k * step;
        if (j < n) {
          if (PAIRS == kNoPairs) elements(raw[PAIRS == kNoPairs ? k : 0], t + j, j, x[0]);
          store(t + j, x[PAIRS == kNoPairs ? 0 : k]);
        }
      }
      for (int j = first + kKept * step; j < n; j += step) {
        float y[kUnit];
        elements(ask(t + j), t + j, j, y);
        store(t + j, y);
      }
      // (every lane has read the scale that was)
      if (TEAM == 1) __syncwarp();
      if (me == 0) *scale_at = scale;
    }
  }
}

template <int TEAM>
cudaError_t launch(const RotaryArgs& a, bool neighbours, cudaStream_t stream) {
  // tokens of a team: so that there are enough teams to fill the GPU
  const int64_t work = (int64_t)a.T * 2 * a.k_heads, teams = 16384 / TEAM;
  const int part = (int)std::min<int64_t>(kMostTokens, std::max<int64_t>(1, work / teams));
  // heads of k that share the angles: as long as the runs of full pages are still one a team
  // and SM (GB300, pages of 64 tokens of 128 elements, all heads at once against one: 4 heads of
  // 900 tokens 34 and 23 us, of 9216 69 and 80; 8 heads of 2997 47 and 41 (37 by this rule), of
  // 23998 220 and 278)
  const int64_t runs = std::max<int64_t>(1, a.T >> a.page_shift);
  const int at_once =
      a.rot == 0 ? 1
                 : (int)std::min<int64_t>(std::min(kMostHeads, a.k_heads),
                                          std::max<int64_t>(1, runs * a.k_heads / 152));
  void (*kernel)(RotaryArgs, int, int) = a.rot == 0   ? page_write_kernel<kNoPairs, TEAM>
                                    : neighbours ? page_write_kernel<kNeighbours, TEAM>
                                                 : page_write_kernel<kHalves, TEAM>;
  const int64_t of_block = (int64_t)part * (kWarps / TEAM);   // tokens
  return launch_kernel(true, dim3((unsigned)((a.T + of_block - 1) / of_block),
                            (a.k_heads + at_once - 1) / at_once + a.k_heads),
                       dim3(32 * kWarps), 0, stream, kernel, a, part, at_once);
}

}  // namespace

int launch_page_write(const RotaryArgs& a, bool neighbours, cudaStream_t stream) {
  const int units = a.head_dim / kUnit << a.page_shift;   // of a full page
  const cudaError_t e =
      units <= 32 * kKept ? launch<1>(a, neighbours, stream) : launch<4>(a, neighbours, stream);
  if (e != cudaSuccess) return -3;
  if (a.q_heads == 0) return 0;
  RotaryArgs q = a;
  q.k_heads = 0;
  q.beside = true;
  return launch_rotary(q, 0, neighbours, stream);
}

}  // namespace moe
