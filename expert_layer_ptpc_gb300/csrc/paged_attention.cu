// Attention of one new token per context over the paged key-value cache.
//
//   s_j = scale q . k_j,  m = max_j s_j,  l = sum_j exp(s_j - m),
//   out = sum_j exp(s_j - m) v_j / l,  lse = m + ln l
//
// One pass over the tokens with a running maximum: when a new maximum
// arrives, the sum and the accumulator are scaled by exp(old - new). One block
// per (context, query head); its warps take tokens in turn, a lane holds
// head_dim / 32 elements, and the warps' (m, l, acc) are joined at the end.
#include <cmath>

#include "attention.h"
#include "common.cuh"
#include "internal.h"

#include <cuda_fp16.h>

namespace moe {

namespace {

constexpr int kWarps = 8;

template <bool E4M3, int N>
__device__ __forceinline__ void load_row(const void* base, int64_t row, int head_dim, int lane,
                                         float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const int64_t at = row * head_dim + 64 * (i / 2) + 2 * lane;
    if (E4M3) {
      const uint16_t c = *reinterpret_cast<const uint16_t*>(static_cast<const uint8_t*>(base) + at);
      uint32_t h;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      x[i] = f.x;
      x[i + 1] = f.y;
    } else {
      const uint32_t w =
          *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(base) + at);
      x[i] = __uint_as_float(w << 16);
      x[i + 1] = __uint_as_float(w & 0xffff0000u);
    }
  }
}

template <bool E4M3, int D>
__global__ void __launch_bounds__(kWarps * 32) paged_attention_kernel(
    const CacheView c, const uint16_t* __restrict__ q, int64_t q_stride, int q_heads,
    const int32_t* __restrict__ lengths, float scale, int window, uint16_t* __restrict__ out,
    float* __restrict__ lse) {
  constexpr int N = D / 32;
  __shared__ float sm[kWarps], sl[kWarps], sacc[kWarps][D];
  const int b = blockIdx.x, h = blockIdx.y;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int kv = h / (q_heads / c.heads);
  const int64_t top = (int64_t)c.max_pages << c.page_shift;
  const int length = lengths[b];
  const int end = (int)min((int64_t)max(length, 0), top);
  const int begin = window > 0 ? max(length - window, 0) : 0;
  float qv[N], acc[N];
  load_row<false>(q + b * q_stride, h, D, lane, qv);
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = 0.f;
  float m = -INFINITY, l = 0.f;
  for (int64_t j = begin + warp; j < end; j += kWarps) {
    const int32_t entry = c.table[b * c.table_stride + (j >> c.page_shift)];
    if ((uint32_t)entry >= (uint32_t)c.pages) continue;
    const int64_t row = (((int64_t)entry * c.heads + kv) << c.page_shift) +
                        (j & ((1 << c.page_shift) - 1));
    float k[N], v[N];
    load_row<E4M3>(c.k, row, D, lane, k);
    load_row<E4M3>(c.v, row, D, lane, v);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) s = fmaf(qv[i], k[i], s);
    s = warp_sum(s) * scale * (E4M3 ? c.k_scale[row] : 1.f);
    const float next = fmaxf(m, s);
    const float old = m == -INFINITY ? 0.f : expf(m - next);
    const float p = s == -INFINITY ? 0.f : expf(s - next);
    const float pv = p * (E4M3 ? c.v_scale[row] : 1.f);
    l = l * old + p;
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = fmaf(pv, v[i], acc[i] * old);
    m = next;
  }
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    sacc[warp][64 * (i / 2) + 2 * lane] = acc[i];
    sacc[warp][64 * (i / 2) + 2 * lane + 1] = acc[i + 1];
  }
  __syncthreads();
  float top_m = -INFINITY, total = 0.f;
  for (int w = 0; w < kWarps; ++w) top_m = fmaxf(top_m, sm[w]);
  for (int w = 0; w < kWarps; ++w)
    total += sm[w] == -INFINITY ? 0.f : sl[w] * expf(sm[w] - top_m);
  for (int d = threadIdx.x; d < D; d += kWarps * 32) {
    float sum = 0.f;
    for (int w = 0; w < kWarps; ++w)
      if (sm[w] != -INFINITY) sum += sacc[w][d] * expf(sm[w] - top_m);
    const __nv_bfloat16 y = __float2bfloat16_rn(total == 0.f ? 0.f : sum / total);
    out[((int64_t)b * q_heads + h) * D + d] = *reinterpret_cast<const uint16_t*>(&y);
  }
  if (lse != nullptr && threadIdx.x == 0)
    lse[(int64_t)b * q_heads + h] = top_m + logf(total);
}

}  // namespace

size_t paged_attention_ws_bytes(int, int, int, int) { return 256; }

int launch_paged_attention(const CacheView& c, const uint16_t* q, int64_t q_stride, int batch,
                           int q_heads, const int32_t* lengths, float scale, int window,
                           uint16_t* out, float* lse, void*, cudaStream_t stream) {
  const dim3 grid(batch, q_heads);
  auto go = [&](auto kernel) {
    kernel<<<grid, kWarps * 32, 0, stream>>>(c, q, q_stride, q_heads, lengths, scale, window, out,
                                             lse);
  };
  if (c.e4m3) {
    if (c.head_dim == 64) go(paged_attention_kernel<true, 64>);
    else if (c.head_dim == 128) go(paged_attention_kernel<true, 128>);
    else go(paged_attention_kernel<true, 256>);
  } else {
    if (c.head_dim == 64) go(paged_attention_kernel<false, 64>);
    else if (c.head_dim == 128) go(paged_attention_kernel<false, 128>);
    else go(paged_attention_kernel<false, 256>);
  }
  return cudaGetLastError() == cudaSuccess ? 0 : -3;
}

}  // namespace moe
