// Block tables and slot maps of a serving step, from request lengths.
//
//   leaving (n_b < 0):  the pages of its h_b tokens go back onto the stack
//   need_b = ceil((h_b + n_b) / page) - ceil(h_b / page)
//   A_b = sum_{i <= b} need_i,  O_b = sum_{i <= b} n_i      (requests that fit the table)
//   served_b: A_b <= F and O_b <= rows      (F pages on the stack, those given back included)
//   page number k of the step is stack[F - 1 - k]; token t of request b lies at slot
//   page(t / page) * page + t % page.
//
// Integers, a few bytes a token and a request: the time is latency, two or three
// dependent reads of memory and a scan. So one launch, and no CTA waits for another:
// each works out the sums over the whole batch for itself (at most 4096 requests, in
// shared memory), puts the pages given back onto the stack itself (all write the same
// values) and reads them behind its own barrier; the tokens and the tables' new
// entries are shared out.
// GB300, in a graph: 128 requests of one token 9.8 us; 301 prompts of up to 110 tokens
// (16384 rows, 16 CTAs) 13.3 us. A call costs the host 24 us.
#include <algorithm>
#include <climits>

#include "attention.h"
#include "common.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kTokens = 2 * kThreads;    // of a CTA, when there are enough
constexpr int kMaxCtas = 64;

struct Sums {
  int64_t back, need, tokens;
};
__device__ __forceinline__ Sums operator+(const Sums& a, const Sums& b) {
  return {a.back + b.back, a.need + b.need, a.tokens + b.tokens};
}
__device__ __forceinline__ Sums from_below(const Sums& a, int o) {
  return {__shfl_up_sync(0xffffffffu, a.back, o), __shfl_up_sync(0xffffffffu, a.need, o),
          __shfl_up_sync(0xffffffffu, a.tokens, o)};
}
__device__ __forceinline__ int clip(int64_t v) { return (int)min(v, (int64_t)INT_MAX); }

__global__ void __launch_bounds__(kThreads) kv_plan_kernel(const PlanArgs a) {
  extern __shared__ int smem[];
  int* const held = smem;                 // [batch] tokens held
  int* const grown = held + a.batch;      // [batch] new tokens of a request that is served, else 0
  int* const back = grown + a.batch;      // [batch] pages given back; then: by those before it
  int* const start = back + a.batch;      // [batch] its first token of the step
  int* const first = start + a.batch;     // [batch] its first page of the step
  __shared__ Sums warp_sums[kWarps];
  __shared__ int taken, total, waiting;   // pages and tokens served, requests that were not
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int page = 1 << a.page_shift;
  const int64_t room = min((int64_t)a.max_pages << a.page_shift, (int64_t)INT_MAX);
  const int stacked = min(max(a.state[a.batch], 0), a.pages);
  auto pages_of = [&](int64_t tokens) -> int64_t { return (tokens + page - 1) >> a.page_shift; };
  auto valid = [&](int32_t p) { return (uint32_t)p < (uint32_t)a.pages; };

  if (threadIdx.x == 0) taken = total = waiting = 0;
  for (int b = threadIdx.x; b < a.batch; b += kThreads) {
    held[b] = a.state[b];
    grown[b] = a.new_tokens[b];
  }
  __syncthreads();
  // pages that a leaving request's table holds
  auto pages_back = [&](int b) -> int {
    return grown[b] < 0 && held[b] > 0 ? (int)min(pages_of(held[b]), (int64_t)a.max_pages) : 0;
  };
  for (int b = warp; b < a.batch; b += kWarps) {
    const int n = pages_back(b);
    int count = 0;
    for (int i = lane; i < n; i += 32) count += valid(a.table[b * a.table_stride + i]);
    if (n > 0) count = __reduce_add_sync(0xffffffffu, count);
    if (lane == 0) back[b] = count;
  }
  __syncthreads();

  // sums over the requests before: each thread has a run of them
  const int per = (a.batch + kThreads - 1) / kThreads;
  const int b0 = threadIdx.x * per, b1 = min(a.batch, b0 + per);
  auto fits = [&](int b) {
    return grown[b] >= 0 && held[b] >= 0 && (int64_t)held[b] + grown[b] <= room;
  };
  auto of = [&](int b) -> Sums {
    Sums s = {back[b], 0, 0};
    if (fits(b)) {
      s.need = pages_of((int64_t)held[b] + grown[b]) - pages_of(held[b]);
      s.tokens = grown[b];
    }
    return s;
  };
  Sums mine = {0, 0, 0};
  for (int b = b0; b < b1; ++b) mine = mine + of(b);
  Sums up = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Sums v = from_below(up, o);
    if (lane >= o) up = up + v;
  }
  if (lane == 31) warp_sums[warp] = up;
  __syncthreads();
  Sums run = {up.back - mine.back, up.need - mine.need, up.tokens - mine.tokens};
  int64_t backs = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) run = run + warp_sums[w];
    backs += warp_sums[w].back;
  }
  // (a stack that holds a page twice can overflow: what lies past its end is dropped)
  const int free = (int)min((int64_t)stacked + backs, (int64_t)a.pages);
  int lost = 0;
  for (int b = b0; b < b1; ++b) {
    const Sums s = of(b), to = run + s;
    const bool ok = fits(b), served = ok && to.need <= free && to.tokens <= a.rows;
    if (served) {
      atomicMax(&taken, (int)to.need);
      atomicMax(&total, (int)to.tokens);
    }
    lost += grown[b] > 0 && !served;
    back[b] = clip(run.back);
    start[b] = clip(run.tokens);
    first[b] = clip(run.need);
    run = to;
    if (!served && grown[b] > 0) grown[b] = 0;
  }
  if (lost > 0) atomicAdd(&waiting, lost);
  __syncthreads();

  // the pages given back, onto the stack
  for (int b = warp; b < a.batch; b += kWarps) {
    const int n = pages_back(b);
    int64_t to = (int64_t)stacked + back[b];
    for (int i0 = 0; i0 < n; i0 += 32) {
      const int32_t p = i0 + lane < n ? a.table[b * a.table_stride + i0 + lane] : -1;
      const unsigned some = __ballot_sync(0xffffffffu, valid(p));
      const int64_t at = to + __popc(some & lanemask_lt());
      if (valid(p) && at < a.pages) a.stack[at] = p;
      to += __popc(some);
    }
  }
  __syncthreads();
  // page number k of the step
  auto page_at = [&](int64_t k) -> int32_t {
    const int64_t at = free - 1 - k;
    return at >= 0 ? a.stack[at] : -1;
  };

  // the tables' new entries, a warp a request
  for (int b = blockIdx.x * kWarps + warp; b < a.batch; b += gridDim.x * kWarps) {
    if (grown[b] <= 0) continue;
    const int64_t have = pages_of(held[b]), need = pages_of((int64_t)held[b] + grown[b]) - have;
    for (int64_t i = lane; i < need; i += 32)
      a.table[b * a.table_stride + have + i] = page_at(first[b] + i);
  }
  // the tokens: the last request that starts at or before one
  for (int64_t t = blockIdx.x * kThreads + threadIdx.x; t < a.rows; t += gridDim.x * kThreads) {
    int32_t slot = -1;
    int at = 0;
    if (t < total) {
      int lo = 0, hi = a.batch;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= t) lo = mid; else hi = mid;
      }
      at = held[lo] + (int)(t - start[lo]);
      const int64_t have = pages_of(held[lo]), i = at >> a.page_shift;
      const int32_t p = i < have ? a.table[lo * a.table_stride + i] : page_at(first[lo] + i - have);
      slot = valid(p) ? (p << a.page_shift) + (at & (page - 1)) : -1;
    }
    a.slots[t] = slot;
    for (int x = 0; x < a.axes; ++x) a.positions[(int64_t)x * a.rows + t] = at;
  }
  if (blockIdx.x == 0) {
    for (int b = threadIdx.x; b < a.batch; b += kThreads) {
      a.offsets[b + 1] = min(clip((int64_t)start[b] + max(grown[b], 0)), total);
      a.state_out[b] = grown[b] < 0 ? 0 : held[b] + grown[b];
    }
    if (threadIdx.x == 0) {
      a.offsets[0] = 0;
      a.state_out[a.batch] = free - taken;
      a.refused[0] = waiting;
    }
  }
}

}  // namespace

int launch_kv_plan(const PlanArgs& a, cudaStream_t stream) {
  const int smem = 5 * a.batch * (int)sizeof(int);   // at most 80 KB
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(kv_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
          cudaSuccess)
    return -3;
  const int ctas = std::min(kMaxCtas, a.rows / kTokens + 1);
  const cudaError_t e = launch_kernel(true, dim3(ctas), dim3(kThreads), smem, stream,
                                      kv_plan_kernel, a);
  return e == cudaSuccess ? 0 : -3;
}

}  // namespace moe
