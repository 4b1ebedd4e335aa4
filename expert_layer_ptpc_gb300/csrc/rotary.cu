// Rotary positions with several axes, and the key-value cache's write, in one
// pass over q, k and v ("Ultimate Latency Optimization of Qwen3 and Qwen3-VL
// on AMD MI300X Series": fused MRoPE of q and k; FP8 cache types).
//
//   pair i of a head:  a = 2 pi frac(p turns[i] / 2^64),  p = positions[axis_i, t]
//   y1 = x1 cos a - x2 sin a,   y2 = x2 cos a + x1 sin a
//   cache row (e4m3):  s = fp32(max(amax, 1e-12) / 448),  q = e4m3(fp32(y / s))
//
// The angle. A frequency is kept as a 64-bit fraction of a turn, so p * turns
// wraps modulo 2^64 exactly as the angle wraps modulo a turn: the integer
// product is the reduced angle, for any 32-bit position, without fp64 or an
// argument reduction. Its upper 32 bits, as a signed fraction in [-1/2, 1/2) turns,
// are rounded to fp32 (by at most 2^-26 turns, a step of fp32 below 1/2 being 2^-25)
// and go to sincospif.
//
// Every element is read once and written once: the kernel is bound by memory
// (4 bytes moved per element of q against 3 flops). A warp takes one token and
// a run of its heads. It works out the token's cosines together, two pairs a lane
// for 128 elements, and every lane keeps the 8 that its elements need in
// registers over all the heads. A lane's unit of a head is two runs of 8 elements,
// half a region apart, so that the lanes' 16-byte accesses are contiguous; the
// next units are in flight while one is used. A cache head is 4, 8 or 16 units,
// hence that many neighbouring lanes, and its row maximum is a shuffle.
// GB300, 8192 tokens of 64 + 4 heads of 128: the rotation 44.7 us (6.4 TB/s of the copy's
// 6.8), with k and v quantised into the cache 47.2 us (6.2 TB/s). 16001 tokens' keys and
// values alone, 8 heads: 19.9 us into an e4m3 cache (4.4 TB/s), 18.5 into a bf16 one
// (6.3 TB/s).
#include <algorithm>

#include "attention.h"
#include "common.cuh"
#include "internal.h"
#include "rotary.cuh"

namespace moe {

namespace {

constexpr int kWarps = 8;
// Blocks of an SM: 32 warps of 64 registers a lane. A lane's units travel through
// shared memory (cp.async, each lane reads back its own), so that more of them are
// in flight than registers would hold. (GB300, 8192 tokens of 64 + 4 heads of 128, the
// rotation and the fused write, one after the other in one run: 44.1 and 46.5 us with
// three units in flight; in registers, two and one, 45.9 and 51.8, and more of them spill.
// As it is, the bf16 caches' fused writes spill 16 bytes, the others nothing.)
constexpr int kBlocks = 4;
constexpr int kAhead = 3;     // units of a lane in flight

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// v / s rounded to nearest, for many v and one s: with y = 1 / s rounded to
// nearest and q = v y within a unit in the last place of v / s, q + y (v - s q)
// with fused products is v / s rounded to nearest (Markstein 1990), where nothing
// under- or overflows. Here s >= 2^-49 and y is normal, and quotients below
// 2^-10 become the code 0 whatever their last bits. The product v y alone can be
// up to 1.5 units off, which the theorem does not cover; so it was tried for all 2^23
// mantissas of s, each with the 9 v around each of the 16 ties between codes and 100
// others: 2 billion quotients, all rounded to nearest.
__device__ __forceinline__ float quotient(float v, float s, float y) {
  const float q = v * y;
  return fmaf(-fmaf(s, q, -v), y, q);   // (this order keeps the sign of a zero)
}

__device__ __forceinline__ uint2 codes8(const float* v, float s, float y) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint16_t lo =
        f32x2_to_e4m3x2(quotient(v[4 * i], s, y), quotient(v[4 * i + 1], s, y));
    const uint16_t hi =
        f32x2_to_e4m3x2(quotient(v[4 * i + 2], s, y), quotient(v[4 * i + 3], s, y));
    w[i] = (uint32_t)lo | ((uint32_t)hi << 16);
  }
  return make_uint2(w[0], w[1]);
}

enum Sink { kSinkTensors = 0, kSinkE4m3 = 1, kSinkBf16 = 2 };

// A token's heads are q's, then k's, then (with a cache) v's. Warp w of the grid
// takes heads [part * per_warp, ...) of token w / parts, part = w % parts.
template <int SINK, int PAIRS>
__global__ void __launch_bounds__(kWarps * 32, kBlocks)
    rotary_kernel(const RotaryArgs a, int parts, int per_warp) {
  constexpr bool NEIGHBOURS = PAIRS == kNeighbours;
  // the warps' units in flight, and the (cos, sin) of their tokens' pairs
  extern __shared__ __align__(16) uint8_t smem[];
  uint8_t* const flight = smem + (threadIdx.x >> 5) * (kAhead * 1024);
  float2* const turns = reinterpret_cast<float2*>(smem + kWarps * kAhead * 1024);
  if (!a.beside) {
    pdl_wait();
    pdl_launch_dependents();
  } else if (blockIdx.x == gridDim.x - 1) {
    // (what q depends on had ended when the launch before this one began; the last block
    // sees that launch out, and without a word to the next that waits for all of this one)
    pdl_wait();
  }
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int t = (int)(w / parts);
  if (t >= a.T) return;
  const int units = a.head_dim / kUnit;              // of a head: lanes
  const int at_once = 32 / units;                    // heads
  const int u = lane % units;
  const int heads = a.q_heads + (SINK == kSinkTensors ? a.k_heads : 2 * a.k_heads);
  const int begin = (int)(w - (int64_t)t * parts) * per_warp;
  const int end = min(heads, begin + per_warp);
  const int mine = lane < at_once * units ? begin + lane / units : end;   // first head
  const int rot_units = PAIRS == kNoPairs ? 0 : a.rot / kUnit;
  const int32_t slot = SINK == kSinkTensors ? -1 : a.slots[t];
  const bool kept = SINK != kSinkTensors && (uint32_t)slot < a.cache_slots;

  // the lane's two runs of 8 elements in a rotated head, and in one of v
  const bool rotates = u < rot_units;
  const int from = rotates ? 0 : a.rot, region = rotates ? a.rot : a.head_dim - a.rot;
  const int run0 = from + 8 * (rotates ? u : u - rot_units), run1 = run0 + region / 2;
  const int v_run0 = 8 * u, v_run1 = v_run0 + a.head_dim / 2;
  const int q_end = a.q_heads, k_end = q_end + a.k_heads;

  // (keys and values of a token without a slot are read all the same: the
  // loads need not wait for the slot)
  auto source = [&](int head) -> const uint16_t* {
    if (PAIRS != kNoPairs && head < q_end) return a.q + t * a.q_stride + head * a.head_dim;
    if (head < k_end) return a.k + t * a.k_stride + (head - q_end) * a.head_dim;
    return a.v + t * a.v_stride + (head - k_end) * a.head_dim;
  };
  // A unit goes to shared memory and back to the lane that asked for it: 32
  // bytes a lane, in flight without registers.
  auto load = [&](int step) {
    const int head = mine + step * at_once;
    const uint32_t to = smem_u32(flight) + (step % kAhead) * 1024 + lane * 16;
    if (head < end) {
      const uint16_t* src = source(head);
      const bool is_v = SINK != kSinkTensors && head >= k_end;
      cp_async_16(to, src + (is_v ? v_run0 : run0));
      cp_async_16(to + 512, src + (is_v ? v_run1 : run1));
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) load(i);

  // cosines of the token's pairs
  float2 cs[8];
  if (PAIRS != kNoPairs) {
    float2* const table = turns + (threadIdx.x >> 5) * (a.rot / 2);
    for (int p = lane; p < a.rot / 2; p += 32) {
      table[p] = turn_of(a, t, a.turns[p], a.pair_axis[p]);
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int p = pair_of<PAIRS>(u, j, a.rot);
      cs[j] = rotates ? table[p] : make_float2(1.f, 0.f);
    }
  }

  const int64_t row0 = ((int64_t)(slot >> a.page_shift) * a.k_heads << a.page_shift) +
                       (slot & ((1 << a.page_shift) - 1));   // of kv head 0
  const int steps = (end - begin + at_once - 1) / at_once;
  for (int step = 0; step < steps; ++step) {
    const int head = mine + step * at_once;
    const bool is_v = SINK != kSinkTensors && head >= k_end;
    asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
    float x[kUnit];
    const uint8_t* const unit = flight + (step % kAhead) * 1024 + lane * 16;
    unpack8(*reinterpret_cast<const uint4*>(unit), x);
    unpack8(*reinterpret_cast<const uint4*>(unit + 512), x + 8);
    load(step + kAhead);
    if (PAIRS != kNoPairs && rotates && !is_v) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        turn_pair(cs[j], NEIGHBOURS ? x[2 * j] : x[j], NEIGHBOURS ? x[2 * j + 1] : x[8 + j]);
    }
    const int o0 = is_v ? v_run0 : run0, o1 = is_v ? v_run1 : run1;
    uint16_t* dst = nullptr;
    if (PAIRS != kNoPairs && head < end) {
      if (head < q_end) dst = a.q_out + t * a.q_out_stride + head * a.head_dim;
      else if (SINK == kSinkTensors)
        dst = a.k_out + t * a.k_out_stride + (head - q_end) * a.head_dim;
    }
    if (dst != nullptr) {
      *reinterpret_cast<uint4*>(dst + o0) = pack8(x);
      *reinterpret_cast<uint4*>(dst + o1) = pack8(x + 8);
    }
    // (the warp's heads of this step, all q's: nothing for the cache)
    if (SINK == kSinkTensors || begin + (step + 1) * at_once <= q_end) continue;

    float amax = 0.f;
    if (SINK == kSinkE4m3) {
#pragma unroll
      for (int j = 0; j < kUnit; ++j) amax = fmaxf(amax, fabsf(x[j]));
      for (int o = units >> 1; o > 0; o >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    }
    if (head < q_end || head >= end || !kept) continue;
    const int kv_head = is_v ? head - k_end : head - q_end;
    const int64_t row = row0 + ((int64_t)kv_head << a.page_shift);
    if (SINK == kSinkE4m3) {
      const float s = __fdiv_rn(fmaxf(amax, 1e-12f), 448.0f), y = __frcp_rn(s);
      uint8_t* out = static_cast<uint8_t*>(is_v ? a.cache_v : a.cache_k) + row * a.head_dim;
      *reinterpret_cast<uint2*>(out + o0) = codes8(x, s, y);
      *reinterpret_cast<uint2*>(out + o1) = codes8(x + 8, s, y);
      if (u == 0) (is_v ? a.v_scale : a.k_scale)[row] = s;
    } else {
      uint16_t* out = static_cast<uint16_t*>(is_v ? a.cache_v : a.cache_k) + row * a.head_dim;
      *reinterpret_cast<uint4*>(out + o0) = pack8(x);
      *reinterpret_cast<uint4*>(out + o1) = pack8(x + 8);
    }
  }
}

}  // namespace

int launch_rotary(const RotaryArgs& a, int sink, bool neighbours, cudaStream_t stream) {
  const int heads = a.q_heads + (sink == kSinkTensors ? a.k_heads : 2 * a.k_heads);
  const int at_once = 32 / (a.head_dim / kUnit);
  const int steps = (heads + at_once - 1) / at_once;   // of a warp that has all heads
  // Steps of a warp: so many that the work fills the GPU three times over (152 SMs
  // with 32 warps each; the rotation above took 44.1 us, 45.8 with all 17 steps of a
  // token in one warp, the last warps being few); but up to 8, as long as it is
  // filled once (4099 tokens of 18 heads of 256 take 14.1 us in steps of 5 and 4, 16.6
  // in steps of 2: each warp works out the cosines anew); at least one.
  const int64_t fill = 152 * 32, work = (int64_t)a.T * steps;
  const int most = (int)std::min<int64_t>(
      steps, std::max<int64_t>({1, work / (3 * fill), std::min<int64_t>(8, work / fill)}));
  const int even = (steps + most - 1) / most;          // warps of a token
  const int take = (steps + even - 1) / even;
  const int per_warp = take * at_once;
  const int parts = (heads + per_warp - 1) / per_warp;
  const int64_t blocks = ((int64_t)parts * a.T + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffff) return -2;
  void (*kernel)(RotaryArgs, int, int) = nullptr;
  if (sink == kSinkTensors)
    kernel = neighbours ? rotary_kernel<kSinkTensors, kNeighbours>
                        : rotary_kernel<kSinkTensors, kHalves>;
  else if (a.rot == 0)   // keys and values as they are
    kernel = sink == kSinkE4m3 ? rotary_kernel<kSinkE4m3, kNoPairs>
                               : rotary_kernel<kSinkBf16, kNoPairs>;
  else if (sink == kSinkE4m3)
    kernel = neighbours ? rotary_kernel<kSinkE4m3, kNeighbours> : rotary_kernel<kSinkE4m3, kHalves>;
  else
    kernel = neighbours ? rotary_kernel<kSinkBf16, kNeighbours> : rotary_kernel<kSinkBf16, kHalves>;
  const size_t smem = (size_t)kWarps * (kAhead * 1024 + (a.rot / 2) * sizeof(float2));
  const cudaError_t e = launch_kernel(true, dim3((unsigned)blocks), dim3(kWarps * 32), smem,
                                      stream, kernel, a, parts, per_warp);
  return e == cudaSuccess ? 0 : -3;
}

}  // namespace moe
