// Attention of many new tokens per context over the paged key-value cache.
//
//   s_ij = scale q_i . k_j for the tokens j that row i sees,
//   out_i = sum_j softmax(s_i)_j v_j,  lse_i = ln sum_j exp(s_ij)
//
// A warp takes one query head of one new token, its lanes the head's elements, and
// goes through the context with a running maximum and sum.
#include <algorithm>

#include "attention.h"
#include "common.cuh"
#include "internal.h"

#include <cuda_fp16.h>

namespace moe {

namespace {

constexpr int kWarps = 8;

struct Args {
  CacheView c;
  const uint16_t* q;
  int64_t q_stride, out_stride;
  int rows, q_heads, batch;
  const int32_t *offsets, *lengths;
  float scale;
  int window;
  uint16_t* out;
  float* lse;
};

template <bool E4M3>
__device__ __forceinline__ float element(const void* p, int64_t at) {
  if (E4M3) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;"
        : "=r"(h)
        : "h"((uint16_t)static_cast<const uint8_t*>(p)[at]));
    return __low2float(*reinterpret_cast<const __half2*>(&h));
  }
  return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[at] << 16);
}

template <bool E4M3, int D>
__global__ void __launch_bounds__(kWarps * 32) prompt_attention_kernel(const Args a) {
  constexpr int N = D / 32;
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int row = (int)(w / a.q_heads), h = (int)(w - (int64_t)row * a.q_heads);
  if (row >= a.rows || row >= a.offsets[a.batch]) return;
  int lo = 0, hi = a.batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.offsets[mid] <= row) lo = mid; else hi = mid;
  }
  const int b = lo;
  const int64_t at = (int64_t)a.lengths[b] - (a.offsets[b + 1] - row);   // the token's place
  const int64_t room = (int64_t)a.c.max_pages << a.c.page_shift;
  const int64_t end = min(at + 1, room);
  const int64_t begin = a.window > 0 ? max(at + 1 - a.window, (int64_t)0) : 0;
  const int kv = h / (a.q_heads / a.c.heads);
  float q[N], acc[N], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    q[i] = element<false>(a.q, row * a.q_stride + h * D + lane + 32 * i);
    acc[i] = 0.f;
  }
  for (int64_t j = begin; j < end; ++j) {
    const int32_t entry = a.c.table[b * a.c.table_stride + (j >> a.c.page_shift)];
    if ((uint32_t)entry >= (uint32_t)a.c.pages) continue;
    const int64_t r = (((int64_t)entry * a.c.heads + kv) << a.c.page_shift) +
                      (j & ((1 << a.c.page_shift) - 1));
    const float ks = E4M3 ? a.c.k_scale[r >> a.c.scale_shift] : 1.f;
    const float vs = E4M3 ? a.c.v_scale[r >> a.c.scale_shift] : 1.f;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) s = fmaf(q[i], element<E4M3>(a.c.k, r * D + lane + 32 * i), s);
    s = warp_sum(s) * ks * a.scale;
    const float top = fmaxf(m, s), was = __expf(m - top), p = __expf(s - top);
    m = top;
    l = fmaf(l, was, p);
#pragma unroll
    for (int i = 0; i < N; ++i)
      acc[i] = fmaf(acc[i], was, p * vs * element<E4M3>(a.c.v, r * D + lane + 32 * i));
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const __nv_bfloat16 y = __float2bfloat16_rn(acc[i] * inv);
    a.out[row * a.out_stride + h * D + lane + 32 * i] = *reinterpret_cast<const uint16_t*>(&y);
  }
  if (lane == 0 && a.lse != nullptr)
    a.lse[(int64_t)row * a.q_heads + h] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace

size_t prompt_attention_ws_bytes(int, int, int) { return 16; }

int launch_prompt_attention(const CacheView& c, const uint16_t* q, int64_t q_stride, int rows,
                            int q_heads, const int32_t* offsets, const int32_t* lengths, int batch,
                            float scale, int window, uint16_t* out, int64_t out_stride, float* lse,
                            void*, cudaStream_t stream) {
  Args a{};
  a.c = c;
  a.q = q;
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.rows = rows;
  a.q_heads = q_heads;
  a.batch = batch;
  a.offsets = offsets;
  a.lengths = lengths;
  a.scale = scale;
  a.window = window;
  a.out = out;
  a.lse = lse;
  const int64_t blocks = ((int64_t)rows * q_heads + kWarps - 1) / kWarps;
  void (*kernel)(Args) = nullptr;
  if (c.e4m3)
    kernel = c.head_dim == 64    ? prompt_attention_kernel<true, 64>
             : c.head_dim == 128 ? prompt_attention_kernel<true, 128>
                                 : prompt_attention_kernel<true, 256>;
  else
    kernel = c.head_dim == 64    ? prompt_attention_kernel<false, 64>
             : c.head_dim == 128 ? prompt_attention_kernel<false, 128>
                                 : prompt_attention_kernel<false, 256>;
  const cudaError_t e =
      launch_kernel(true, dim3((unsigned)blocks), dim3(kWarps * 32), 0, stream, kernel, a);
  return e == cudaSuccess ? 0 : -3;
}

}  // namespace moe
