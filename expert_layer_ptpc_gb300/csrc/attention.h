// Internal launchers of the attention entry points (api_attention.cu checks
// their arguments). Each returns a moe_status.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace moe {

// q, k and v of T tokens, the rotation, and where the results go: bf16
// tensors (sink 0), or q to a tensor and k, v to a cache (sink 1: e4m3, 2:
// bf16). Strides count elements between tokens.
struct RotaryArgs {
  const uint16_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  uint16_t *q_out, *k_out;
  int64_t q_out_stride, k_out_stride;
  const int32_t* positions;
  const uint64_t* turns;
  const uint8_t* pair_axis;
  int axes, rot, inverse;
  int T, q_heads, k_heads, head_dim;
  const int32_t* slots;
  void *cache_k, *cache_v;
  float *k_scale, *v_scale;
  uint32_t cache_slots;
  int page_shift;
};
int launch_rotary(const RotaryArgs& a, int sink, bool neighbours, cudaStream_t stream);

// A checked cache and the block table of a batch of contexts.
struct CacheView {
  const void *k, *v;
  const float *k_scale, *v_scale;
  int pages, heads, page_shift, head_dim;
  bool e4m3;
  const int32_t* table;
  int64_t table_stride;
  int max_pages;
};

int launch_kv_read(const CacheView& c, const int32_t* offsets, int batch, int64_t rows,
                   uint16_t* k_out, uint16_t* v_out, cudaStream_t stream);

size_t paged_attention_ws_bytes(int heads, int head_dim, int q_heads);
int launch_paged_attention(const CacheView& c, const uint16_t* q, int64_t q_stride, int batch,
                           int q_heads, const int32_t* lengths, float scale, int window,
                           uint16_t* out, float* lse, void* ws, cudaStream_t stream);

}  // namespace moe
