// C ABI of the attention operators: argument checks in front of the kernels
// of rotary.cu, kv_read.cu and paged_attention.cu. Declared in moe_ptpc.h.
#include <cmath>

#include "../../include/moe_ptpc.h"
#include "attention.h"

namespace moe {

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool good16(const void* p) { return p != nullptr && aligned16(p); }

// A [T, heads, head_dim] bf16 tensor with `stride` elements between tokens.
bool good_heads(const void* p, int64_t stride, int heads, int head_dim) {
  return good16(p) && stride % 8 == 0 && stride >= (int64_t)heads * head_dim;
}

int log2_of(int v) {
  int s = 0;
  while ((1 << s) < v) ++s;
  return s;
}

int check_plan(const moe_rotary_plan* p, const int32_t* positions, int head_dim) {
  if (p == nullptr || p->turns == nullptr || p->pair_axis == nullptr || positions == nullptr)
    return MOE_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(p->turns) & 7u) != 0 ||
      (reinterpret_cast<uintptr_t>(positions) & 3u) != 0)
    return MOE_ERR_INVALID_ARG;
  if (p->axes < 1 || p->axes > 8 || (p->neighbours != 0 && p->neighbours != 1) ||
      p->rot_dim <= 0 || p->rot_dim % 16 != 0 || p->rot_dim > head_dim)
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

int check_cache(const moe_kv_cache* c) {
  if (c == nullptr || c->pages <= 0 || c->heads <= 0 || c->page_size <= 0 || c->head_dim <= 0)
    return MOE_ERR_INVALID_ARG;
  if (c->dtype != MOE_DTYPE_BF16 && c->dtype != MOE_DTYPE_E4M3) return MOE_ERR_INVALID_ARG;
  if (!good16(c->k) || !good16(c->v)) return MOE_ERR_INVALID_ARG;
  const bool e4m3 = c->dtype == MOE_DTYPE_E4M3;
  if (e4m3 ? !good16(c->k_scale) || !good16(c->v_scale)
           : c->k_scale != nullptr || c->v_scale != nullptr)
    return MOE_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
    return MOE_ERR_UNSUPPORTED;
  if (c->page_size > 1024 || (c->page_size & (c->page_size - 1)) != 0)
    return MOE_ERR_UNSUPPORTED;
  const int64_t slots = (int64_t)c->pages * c->page_size;
  // slots < 2^41 here, so the product with heads cannot be formed blindly
  if (slots >= (int64_t(1) << 31)) return MOE_ERR_UNSUPPORTED;
  if (c->heads >= (1 << 16) || slots * c->heads >= (int64_t(1) << 32) - 1)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

CacheView view_of(const moe_kv_cache& c, const int32_t* table, int64_t table_stride,
                  int max_pages) {
  CacheView v{};
  v.k = c.k;
  v.v = c.v;
  v.k_scale = c.k_scale;
  v.v_scale = c.v_scale;
  v.pages = c.pages;
  v.heads = c.heads;
  v.page_shift = log2_of(c.page_size);
  v.head_dim = c.head_dim;
  v.e4m3 = c.dtype == MOE_DTYPE_E4M3;
  v.table = table;
  v.table_stride = table_stride;
  v.max_pages = max_pages;
  return v;
}

// A token with no page at all needs no table.
int check_table(const int32_t* table, int64_t table_stride, int max_pages) {
  if (max_pages < 0 || table_stride < max_pages) return MOE_ERR_INVALID_ARG;
  if (max_pages > 0 &&
      (table == nullptr || (reinterpret_cast<uintptr_t>(table) & 3u) != 0))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

bool good4(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

void set_cache(RotaryArgs* a, const moe_kv_cache& c, const int32_t* slots) {
  a->slots = slots;
  a->cache_k = c.k;
  a->cache_v = c.v;
  a->k_scale = c.k_scale;
  a->v_scale = c.v_scale;
  a->cache_slots = (uint32_t)((int64_t)c.pages * c.page_size);
  a->page_shift = log2_of(c.page_size);
}

void set_plan(RotaryArgs* a, const moe_rotary_plan& p, const int32_t* positions) {
  a->positions = positions;
  a->turns = p.turns;
  a->pair_axis = p.pair_axis;
  a->axes = p.axes;
  a->rot = p.rot_dim;
}

constexpr int kMaxTokenElements = 65536;

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_rotary(const moe_rotary_plan* plan, const int32_t* positions, int T, int head_dim,
               const uint16_t* q, int64_t q_stride, int q_heads, uint16_t* q_out,
               int64_t q_out_stride, const uint16_t* k, int64_t k_stride, int k_heads,
               uint16_t* k_out, int64_t k_out_stride, int inverse, moe_stream_t stream) {
  if (T < 0 || head_dim <= 0 || q_heads < 1) return MOE_ERR_INVALID_ARG;
  if (k != nullptr && k_heads < 1) return MOE_ERR_INVALID_ARG;
  if (head_dim % 16 != 0 || head_dim > 512) return MOE_ERR_UNSUPPORTED;
  const int64_t kh = k != nullptr ? k_heads : 0;
  if ((q_heads + kh) * head_dim > kMaxTokenElements) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (const int st = check_plan(plan, positions, head_dim)) return st;
  if (!good_heads(q, q_stride, q_heads, head_dim) ||
      !good_heads(q_out, q_out_stride, q_heads, head_dim))
    return MOE_ERR_INVALID_ARG;
  if (k != nullptr && (!good_heads(k, k_stride, k_heads, head_dim) ||
                       !good_heads(k_out, k_out_stride, k_heads, head_dim)))
    return MOE_ERR_INVALID_ARG;
  RotaryArgs a{};
  a.T = T;
  a.head_dim = head_dim;
  a.q = q;
  a.q_stride = q_stride;
  a.q_heads = q_heads;
  a.q_out = q_out;
  a.q_out_stride = q_out_stride;
  a.k = k;
  a.k_stride = k_stride;
  a.k_heads = (int)kh;
  a.k_out = k_out;
  a.k_out_stride = k_out_stride;
  a.inverse = inverse != 0;
  set_plan(&a, *plan, positions);
  return launch_rotary(a, 0, plan->neighbours != 0, stream);
}

int moe_kv_write(const moe_kv_cache* cache, const int32_t* slots, int T, const uint16_t* k,
                 int64_t k_stride, const uint16_t* v, int64_t v_stride, moe_stream_t stream) {
  if (T < 0) return MOE_ERR_INVALID_ARG;
  if (const int st = check_cache(cache)) return st;
  if ((int64_t)cache->heads * cache->head_dim * 2 > kMaxTokenElements)
    return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!good4(slots) || !good_heads(k, k_stride, cache->heads, cache->head_dim) ||
      !good_heads(v, v_stride, cache->heads, cache->head_dim))
    return MOE_ERR_INVALID_ARG;
  RotaryArgs a{};
  a.T = T;
  a.head_dim = cache->head_dim;
  a.k = k;
  a.k_stride = k_stride;
  a.k_heads = cache->heads;
  a.v = v;
  a.v_stride = v_stride;
  set_cache(&a, *cache, slots);
  return launch_rotary(a, cache->dtype == MOE_DTYPE_E4M3 ? 1 : 2, false, stream);
}

int moe_rotary_kv_write(const moe_rotary_plan* plan, const int32_t* positions,
                        const moe_kv_cache* cache, const int32_t* slots, int T,
                        const uint16_t* q, int64_t q_stride, int q_heads, uint16_t* q_out,
                        int64_t q_out_stride, const uint16_t* k, int64_t k_stride,
                        const uint16_t* v, int64_t v_stride, moe_stream_t stream) {
  if (T < 0 || q_heads < 1) return MOE_ERR_INVALID_ARG;
  if (const int st = check_cache(cache)) return st;
  const int d = cache->head_dim;
  if (((int64_t)q_heads + 2 * (int64_t)cache->heads) * d > kMaxTokenElements)
    return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (const int st = check_plan(plan, positions, d)) return st;
  if (!good4(slots) || !good_heads(q, q_stride, q_heads, d) ||
      !good_heads(q_out, q_out_stride, q_heads, d) ||
      !good_heads(k, k_stride, cache->heads, d) || !good_heads(v, v_stride, cache->heads, d))
    return MOE_ERR_INVALID_ARG;
  RotaryArgs a{};
  a.T = T;
  a.head_dim = d;
  a.q = q;
  a.q_stride = q_stride;
  a.q_heads = q_heads;
  a.q_out = q_out;
  a.q_out_stride = q_out_stride;
  a.k = k;
  a.k_stride = k_stride;
  a.k_heads = cache->heads;
  a.v = v;
  a.v_stride = v_stride;
  set_plan(&a, *plan, positions);
  set_cache(&a, *cache, slots);
  return launch_rotary(a, cache->dtype == MOE_DTYPE_E4M3 ? 1 : 2, plan->neighbours != 0, stream);
}

int moe_kv_read(const moe_kv_cache* cache, const int32_t* block_table, int64_t table_stride,
                int max_pages, const int32_t* offsets, int batch, int64_t rows, uint16_t* k_out,
                uint16_t* v_out, moe_stream_t stream) {
  if (batch < 1 || rows < 0) return MOE_ERR_INVALID_ARG;
  if (const int st = check_cache(cache)) return st;
  if (rows >= (int64_t(1) << 31)) return MOE_ERR_UNSUPPORTED;   // offsets are int32
  if (rows == 0) return MOE_OK;
  if (const int st = check_table(block_table, table_stride, max_pages)) return st;
  if (!good4(offsets) || !good16(k_out) || !good16(v_out)) return MOE_ERR_INVALID_ARG;
  return launch_kv_read(view_of(*cache, block_table, table_stride, max_pages), offsets, batch,
                        rows, k_out, v_out, stream);
}

size_t moe_paged_attention_workspace_size(const moe_kv_cache* cache, int batch, int q_heads) {
  if (check_cache(cache) != MOE_OK || batch < 0 || batch > 65535 || q_heads < 1 ||
      q_heads % cache->heads != 0)
    return 0;
  return paged_attention_ws_bytes(cache->heads, cache->head_dim, q_heads);
}

int moe_paged_attention(const moe_kv_cache* cache, const uint16_t* q, int64_t q_stride, int batch,
                        int q_heads, const int32_t* block_table, int64_t table_stride,
                        int max_pages, const int32_t* lengths, float scale, int window,
                        uint16_t* out, float* lse, void* ws, size_t ws_bytes,
                        moe_stream_t stream) {
  if (batch < 0 || q_heads < 1 || window < 0 || !std::isfinite(scale))
    return MOE_ERR_INVALID_ARG;
  if (const int st = check_cache(cache)) return st;
  if (q_heads % cache->heads != 0) return MOE_ERR_INVALID_ARG;
  if (batch > 65535 || q_heads > 65535) return MOE_ERR_UNSUPPORTED;
  if (batch == 0) return MOE_OK;
  if (const int st = check_table(block_table, table_stride, max_pages)) return st;
  if (!good_heads(q, q_stride, q_heads, cache->head_dim) || !good4(lengths) || !good16(out) ||
      (lse != nullptr && !good4(lse)))
    return MOE_ERR_INVALID_ARG;
  if (!good16(ws) || ws_bytes < paged_attention_ws_bytes(cache->heads, cache->head_dim, q_heads))
    return MOE_ERR_WORKSPACE;
  return launch_paged_attention(view_of(*cache, block_table, table_stride, max_pages), q,
                                q_stride, batch, q_heads, lengths, scale, window, out, lse, ws,
                                stream);
}

}  // extern "C"
