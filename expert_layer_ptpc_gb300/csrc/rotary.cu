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
// argument reduction. Its upper 32 bits, as a signed fraction, go to sincospif.
//
// Every element is read once and written once: the kernel is bound by memory
// (4 bytes moved per element of q against 3 flops). A thread owns a unit of
// 16 elements (8 pairs): two 16-byte loads, in flight before the block works
// out the token's cosines, which all heads of the token share through shared
// memory. A cache head is 4, 8 or 16 units, hence that many neighbouring
// lanes of one warp, and its row maximum is a shuffle.
#include <algorithm>

#include "attention.h"
#include "common.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kUnit = 16;   // elements per thread

__device__ __forceinline__ void unpack8(const uint4& raw, float* v) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float* v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint2 codes8(const float* v, float s) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint16_t lo =
        f32x2_to_e4m3x2(__fdiv_rn(v[4 * i], s), __fdiv_rn(v[4 * i + 1], s));
    const uint16_t hi =
        f32x2_to_e4m3x2(__fdiv_rn(v[4 * i + 2], s), __fdiv_rn(v[4 * i + 3], s));
    w[i] = (uint32_t)lo | ((uint32_t)hi << 16);
  }
  return make_uint2(w[0], w[1]);
}

enum Sink { kSinkTensors = 0, kSinkE4m3 = 1, kSinkBf16 = 2 };

// One block: one token's units [chunk * kThreads, ...). A token's units are
// q's heads, then k's, then (with a cache) v's.
template <int SINK, bool NEIGHBOURS>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryArgs a, int chunks) {
  __shared__ float2 turn[256];   // (cos, sin) of pair 8 u + j at j * (rot / 16) + u
  const int t = blockIdx.x / chunks;
  const int unit = (blockIdx.x - t * chunks) * kThreads + threadIdx.x;
  const int per_head = a.head_dim / kUnit;
  const int rot_units = a.rot / kUnit;
  const int head = unit / per_head, u = unit - head * per_head;

  // what this thread's unit belongs to
  const uint16_t* src = nullptr;
  uint16_t* dst = nullptr;       // kSinkTensors and q
  bool rotated = u < rot_units;
  int kv_head = -1;              // cache head, when the unit goes to the cache
  bool is_v = false;
  int32_t slot = -1;
  if (head < a.q_heads) {
    src = a.q + t * a.q_stride + head * a.head_dim;
    dst = a.q_out + t * a.q_out_stride + head * a.head_dim;
  } else if (SINK == kSinkTensors) {
    if (head < a.q_heads + a.k_heads) {
      const int h = head - a.q_heads;
      src = a.k + t * a.k_stride + h * a.head_dim;
      dst = a.k_out + t * a.k_out_stride + h * a.head_dim;
    }
  } else if (head < a.q_heads + 2 * a.k_heads) {
    slot = a.slots[t];
    if ((uint32_t)slot < a.cache_slots) {
      kv_head = head - a.q_heads;
      is_v = kv_head >= a.k_heads;
      if (is_v) kv_head -= a.k_heads;
      src = is_v ? a.v + t * a.v_stride + kv_head * a.head_dim
                 : a.k + t * a.k_stride + kv_head * a.head_dim;
      if (is_v) rotated = false;
    }
  }
  // the unit's two runs of 8 elements
  const bool split = rotated && !NEIGHBOURS;
  const int o0 = split ? 8 * u : kUnit * u;
  const int o1 = split ? a.rot / 2 + 8 * u : kUnit * u + 8;
  uint4 raw0 = make_uint4(0, 0, 0, 0), raw1 = raw0;
  if (src != nullptr) {
    raw0 = *reinterpret_cast<const uint4*>(src + o0);
    raw1 = *reinterpret_cast<const uint4*>(src + o1);
  }
  for (int p = threadIdx.x; p < a.rot / 2; p += kThreads) {
    const int axis = a.pair_axis[p];
    const int32_t pos = axis < a.axes ? a.positions[(int64_t)axis * a.T + t] : 0;
    const uint64_t f = (uint64_t)(int64_t)pos * a.turns[p];
    float s, c;
    sincospif((float)(int32_t)(f >> 32) * 0x1p-31f, &s, &c);
    turn[(p & 7) * rot_units + (p >> 3)] = make_float2(c, a.inverse ? -s : s);
  }
  __syncthreads();

  float x[kUnit];
  unpack8(raw0, x);
  unpack8(raw1, x + 8);
  if (rotated) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 cs = turn[j * rot_units + u];
      float& x1 = NEIGHBOURS ? x[2 * j] : x[j];
      float& x2 = NEIGHBOURS ? x[2 * j + 1] : x[8 + j];
      const float y1 = fmaf(x1, cs.x, -(x2 * cs.y));
      x2 = fmaf(x2, cs.x, x1 * cs.y);
      x1 = y1;
    }
  }

  if (SINK != kSinkTensors && kv_head >= 0) dst = nullptr;
  if (dst != nullptr) {
    *reinterpret_cast<uint4*>(dst + o0) = pack8(x);
    *reinterpret_cast<uint4*>(dst + o1) = pack8(x + 8);
  }
  if (SINK == kSinkTensors) return;

  float amax = 0.f;
  if (SINK == kSinkE4m3) {
#pragma unroll
    for (int j = 0; j < kUnit; ++j) amax = fmaxf(amax, fabsf(x[j]));
    for (int o = per_head >> 1; o > 0; o >>= 1)
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  }
  if (kv_head < 0) return;
  const int64_t row =
      ((int64_t)(slot >> a.page_shift) * a.k_heads + kv_head) * (int64_t(1) << a.page_shift) +
      (slot & ((1 << a.page_shift) - 1));
  if (SINK == kSinkE4m3) {
    const float s = __fdiv_rn(fmaxf(amax, 1e-12f), 448.0f);
    uint8_t* out = static_cast<uint8_t*>(is_v ? a.cache_v : a.cache_k) + row * a.head_dim;
    *reinterpret_cast<uint2*>(out + o0) = codes8(x, s);
    *reinterpret_cast<uint2*>(out + o1) = codes8(x + 8, s);
    if (u == 0) (is_v ? a.v_scale : a.k_scale)[row] = s;
  } else {
    uint16_t* out = static_cast<uint16_t*>(is_v ? a.cache_v : a.cache_k) + row * a.head_dim;
    *reinterpret_cast<uint4*>(out + o0) = pack8(x);
    *reinterpret_cast<uint4*>(out + o1) = pack8(x + 8);
  }
}

}  // namespace

int launch_rotary(const RotaryArgs& a, int sink, bool neighbours, cudaStream_t stream) {
  const int heads = a.q_heads + (sink == kSinkTensors ? a.k_heads : 2 * a.k_heads);
  const int units = heads * (a.head_dim / kUnit);
  const int chunks = (units + kThreads - 1) / kThreads;
  const int64_t blocks = (int64_t)chunks * a.T;
  if (blocks > 0x7fffffff) return -2;
  void (*kernel)(RotaryArgs, int) = nullptr;
  if (sink == kSinkTensors)
    kernel = neighbours ? rotary_kernel<kSinkTensors, true> : rotary_kernel<kSinkTensors, false>;
  else if (sink == kSinkE4m3)
    kernel = neighbours ? rotary_kernel<kSinkE4m3, true> : rotary_kernel<kSinkE4m3, false>;
  else
    kernel = neighbours ? rotary_kernel<kSinkBf16, true> : rotary_kernel<kSinkBf16, false>;
  kernel<<<(unsigned)blocks, kThreads, 0, stream>>>(a, chunks);
  return cudaGetLastError() == cudaSuccess ? 0 : -3;
}

}  // namespace moe
