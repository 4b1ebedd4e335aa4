// What the kernels that rotate heads share: a lane's unit of a head, and a pair's turn.
#pragma once

#include "attention.h"
#include "common.cuh"

namespace moe {

// A lane's unit of a head is two runs of 8 elements, half a region apart (a region is
// the rotated elements, or the others).
constexpr int kUnit = 16;

enum Pairs { kNoPairs = 0, kHalves = 1, kNeighbours = 2 };

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

// (cos, sin) of a pair of token t.
__device__ __forceinline__ float2 turn_of(const RotaryArgs& a, int t, uint64_t turns, int axis) {
  const int32_t pos = axis < a.axes ? a.positions[(int64_t)axis * a.T + t] : 0;
  const uint64_t f = (uint64_t)(int64_t)pos * turns;
  float s, c;
  sincospif((float)(int32_t)(f >> 32) * 0x1p-31f, &s, &c);
  return make_float2(c, a.inverse ? -s : s);
}

// The j-th pair of unit u. Pairs (i, i + rot / 2): element j of the first run with that
// of the second; neighbours: four in each run.
template <int PAIRS>
__device__ __forceinline__ int pair_of(int u, int j, int rot) {
  return PAIRS == kNeighbours ? (j < 4 ? 4 * u + j : rot / 4 + 4 * u + j - 4) : 8 * u + j;
}

__device__ __forceinline__ void turn_pair(const float2 cs, float& x1, float& x2) {
  const float y1 = fmaf(x1, cs.x, -(x2 * cs.y));
  x2 = fmaf(x2, cs.x, x1 * cs.y);
  x1 = y1;
}

}  // namespace moe
