// Reading contexts back from the paged key-value cache: out row r of context
// b is the cache row of token r - offsets[b], as bf16(fp32(code) * scale).
//
// Bound by memory: an e4m3 row is read once (1 byte an element and its scale)
// and written once (2 bytes). A thread owns 16 elements of one row: one
// 16-byte load of codes, two 16-byte stores.
#include "attention.h"
#include "common.cuh"
#include "internal.h"

#include <cuda_fp16.h>

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kUnit = 16;

// Two e4m3 codes (low byte first) as fp32.
__device__ __forceinline__ float2 e4m3x2_to_f32(uint16_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

template <bool E4M3>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(
    const CacheView c, const int32_t* __restrict__ offsets, int batch, int64_t rows,
    uint16_t* __restrict__ k_out, uint16_t* __restrict__ v_out) {
  const int per_row = c.heads * (c.head_dim / kUnit);   // units of one token
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t r = i / per_row;
  if (r >= rows) return;
  const int unit = (int)(i - r * per_row);
  const int head = unit / (c.head_dim / kUnit);
  const int d = (unit - head * (c.head_dim / kUnit)) * kUnit;
  // the context of row r: the last b with offsets[b] <= r
  int lo = 0, hi = batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (offsets[mid] <= r) lo = mid; else hi = mid;
  }
  const int64_t token = r - offsets[lo];
  const int64_t page = token >> c.page_shift;
  int32_t entry = -1;
  if (token >= 0 && r < offsets[lo + 1] && page < c.max_pages)
    entry = c.table[lo * c.table_stride + page];
  const bool here = (uint32_t)entry < (uint32_t)c.pages;
  const int64_t row = (((int64_t)entry * c.heads + head) << c.page_shift) +
                      (token & ((1 << c.page_shift) - 1));
  const int64_t out = (r * c.heads + head) * c.head_dim + d;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    uint4 y[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (here) {
      if (E4M3) {
        const uint8_t* base = static_cast<const uint8_t*>(which ? c.v : c.k);
        const uint4 raw = *reinterpret_cast<const uint4*>(base + row * c.head_dim + d);
        const float s = (which ? c.v_scale : c.k_scale)[row];
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
        uint32_t p[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 f = e4m3x2_to_f32((uint16_t)(w[j >> 1] >> (16 * (j & 1))));
          const __nv_bfloat162 b = __floats2bfloat162_rn(__fmul_rn(f.x, s), __fmul_rn(f.y, s));
          p[j] = *reinterpret_cast<const uint32_t*>(&b);
        }
        y[0] = make_uint4(p[0], p[1], p[2], p[3]);
        y[1] = make_uint4(p[4], p[5], p[6], p[7]);
      } else {
        const uint16_t* base = static_cast<const uint16_t*>(which ? c.v : c.k);
        const uint4* from = reinterpret_cast<const uint4*>(base + row * c.head_dim + d);
        y[0] = from[0];
        y[1] = from[1];
      }
    }
    uint4* to = reinterpret_cast<uint4*>((which ? v_out : k_out) + out);
    to[0] = y[0];
    to[1] = y[1];
  }
}

}  // namespace

int launch_kv_read(const CacheView& c, const int32_t* offsets, int batch, int64_t rows,
                   uint16_t* k_out, uint16_t* v_out, cudaStream_t stream) {
  const int64_t units = rows * c.heads * (c.head_dim / kUnit);
  const int64_t blocks = (units + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffff) return -2;
  if (c.e4m3)
    kv_read_kernel<true><<<(unsigned)blocks, kThreads, 0, stream>>>(c, offsets, batch, rows,
                                                                     k_out, v_out);
  else
    kv_read_kernel<false><<<(unsigned)blocks, kThreads, 0, stream>>>(c, offsets, batch, rows,
                                                                      k_out, v_out);
  return cudaGetLastError() == cudaSuccess ? 0 : -3;
}

}  // namespace moe
