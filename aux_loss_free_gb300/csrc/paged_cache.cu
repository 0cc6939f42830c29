// The paged key/value cache's step plan and its write side (sm_103a).
//
// Relay article ("Una carrera de relevos con GPUs alquiladas entrenó el MoE de 2.7B de
// NanoColibri por $200"), opening section: the model's attention (grouped-query, per-head
// QK-norm) as it is served; the paged cache is this library's own form.
//
// paged_plan_kernel: row starts, block tables, slots and lengths of one step from the
// requests' lengths.  Two prefix sums over the requests decide everything: of the new
// tokens (row starts), and of the pages that each request begins (its place in the pool's
// ring; a request is granted while the sum stays within the pool).  Every CTA repeats both
// sums (at most 4096 requests, 8 bytes each) instead of waiting for another CTA, keeps the
// results in shared memory and then serves its own token rows, so the step is one launch
// without a grid barrier.  A fresh page has exactly one new token at its first position
// (the fresh pages start at or after ctx_len rounded up), so the thread with that token
// writes the table entry: no separate pass over the table.  The call moves a few bytes per
// token; it is bound by the launch and the chain load - sums - search - pool load - store.
//
// paged_append_kernel: one warp per token row; q and k heads normalised in fp32, q to its
// row, k and v to their page.  A copy with a reduction, bound by memory traffic.
#include <cuda_bf16.h>

#include "internal.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr unsigned FULL = 0xFFFFFFFFu;
constexpr int HD = kAttnHeadDim;
constexpr int PLAN_THREADS = 256;

struct PlanParams {
  const int32_t* ctx_len;
  const int32_t* new_len;
  int32_t* table;
  int32_t* pool;
  const int32_t* pool_in;
  int32_t* pool_out;
  int32_t* row_start;
  int32_t* slot_map;
  int32_t* kv_len;
  int32_t* next_ctx;
  int32_t* info;
  int* status;
  int R, T, pages, max_pages, page_shift;
};

// Exclusive sum of v over the block's threads; *total receives the block's sum.
__device__ long long block_exclusive_sum(long long v, long long* warp_sums, long long* total) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  long long inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long up = __shfl_up_sync(FULL, inc, o);
    if (lane >= o) inc += up;
  }
  __syncthreads();  // the previous use of warp_sums is over
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < PLAN_THREADS / 32; ++w) {
    const long long x = warp_sums[w];
    if (w < warp) before += x;
    all += x;
  }
  *total = all;
  return before + inc - v;
}

__global__ void __launch_bounds__(PLAN_THREADS) paged_plan_kernel(const PlanParams p) {
  extern __shared__ int32_t plan_smem[];
  int32_t* const s_row = plan_smem;             // [R + 1] row starts, at most T
  int32_t* const s_ctx = s_row + p.R + 1;       // [R]
  int32_t* const s_first = s_ctx + p.R;         // [R] place of the first fresh page in the ring; -1 = denied
  int32_t* const s_back = s_first + p.R;        // [R] ended: place of its first returned page, counted from count; -1
  __shared__ long long warp_sums[PLAN_THREADS / 32];
  const int tid = threadIdx.x;
  const int page = 1 << p.page_shift;
  const long long cap = (long long)p.max_pages << p.page_shift;
  pdl_wait();
  pdl_trigger();
  const int head_in = p.pool_in[0], count_in = p.pool_in[1];
  const bool pool_ok = head_in >= 0 && head_in < p.pages && count_in >= 0 && count_in <= p.pages;
  const int head = pool_ok ? head_in : 0, count = pool_ok ? count_in : 0;
  bool bad = !pool_ok;

  // This thread's requests: a contiguous run, so that its sums extend the block's.
  const int per = (p.R + PLAN_THREADS - 1) / PLAN_THREADS;
  const int r0 = min(p.R, tid * per), r1 = min(p.R, r0 + per);
  long long rows = 0;
  for (int r = r0; r < r1; ++r) rows += max(p.new_len[r], 0);
  long long all_rows, all_need, all_back;
  const long long row0 = block_exclusive_sum(rows, warp_sums, &all_rows);

  long long need = 0, back = 0, row = row0;
  for (int r = r0; r < r1; ++r) {
    const int c = p.ctx_len[r], n = p.new_len[r];
    s_ctx[r] = c;
    s_row[r] = (int)min(row, (long long)p.T);
    row += max(n, 0);
    const long long end = (long long)c + max(n, 0);
    const bool fits = c >= 0 && end <= cap && (n <= 0 || row <= p.T);
    if (!fits) bad = true;
    const int have = (int)((min(max((long long)c, 0LL), cap) + page - 1) >> p.page_shift);
    if (n > 0 && fits) need += ((end + page - 1) >> p.page_shift) - have;
    if (n < 0) back += have;
  }
  const long long need0 = block_exclusive_sum(need, warp_sums, &all_need);
  const long long back0 = block_exclusive_sum(back, warp_sums, &all_back);

  const bool first_cta = blockIdx.x == 0;
  long long upto = need0, ret = back0, taken = 0, denied = 0;
  row = row0;
  for (int r = r0; r < r1; ++r) {
    const int c = s_ctx[r], n = p.new_len[r];
    row += max(n, 0);
    const long long end = (long long)c + max(n, 0);
    const bool fits = c >= 0 && end <= cap && row <= p.T;
    const int have = (int)((min(max((long long)c, 0LL), cap) + page - 1) >> p.page_shift);
    const long long want = n > 0 && fits ? ((end + page - 1) >> p.page_shift) - have : 0;
    upto += want;
    const bool granted = n > 0 && fits && (want == 0 || upto <= count);
    s_first[r] = granted ? (int)(want ? upto - want : 0) : -1;
    s_back[r] = n < 0 ? (int)min(ret, (long long)p.pages) : -1;
    if (n < 0) ret += have;
    if (granted) taken = max(taken, want ? upto : 0);
    if (n > 0 && !granted) ++denied;
    if (first_cta) {
      p.row_start[r] = s_row[r];
      p.kv_len[r] = granted || n == 0 ? (int)end : 0;
      p.next_ctx[r] = granted ? (int)end : n < 0 ? 0 : c;
    }
  }
  if (tid == 0) s_row[p.R] = (int)min(all_rows, (long long)p.T);
  if (first_cta) {
    // Sum of the denied and the largest granted sum of pages, over the block.
    long long all_denied;
    block_exclusive_sum(denied, warp_sums, &all_denied);
    __shared__ int s_taken;
    if (tid == 0) s_taken = 0;
    __syncthreads();
    if (taken) atomicMax(&s_taken, (int)taken);
    __syncthreads();
    if (tid == 0) {
      const int gone = s_taken;
      // No more than `pages` pages are free: a caller that returns a page twice is told so.
      const long long left = (long long)count - gone + all_back;
      if (count + all_back > p.pages) bad = true;
      p.row_start[p.R] = (int)min(all_rows, (long long)p.T);
      p.pool_out[0] = (int)(((long long)head + gone) % p.pages);
      p.pool_out[1] = (int)min(left, (long long)p.pages);
      p.info[0] = (int)min(all_rows, (long long)p.T);
      p.info[1] = gone;
      p.info[2] = (int)min(all_back, (long long)p.pages);
      p.info[3] = (int)all_denied;
    }
  }
  __syncthreads();

  // The rows' slots; a token at the first position of a page writes its table entry.
  const int used = s_row[p.R];
  for (int t = blockIdx.x * PLAN_THREADS + tid; t < p.T; t += gridDim.x * PLAN_THREADS) {
    int slot = -1;
    if (t < used) {
      int lo = 0, hi = p.R;  // the last r with s_row[r] <= t: s_row[lo] <= t < s_row[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_row[mid] <= t) lo = mid;
        else hi = mid;
      }
      const int first = s_first[lo];
      if (first >= 0) {
        const int c = s_ctx[lo], pos = c + (t - s_row[lo]), j = pos >> p.page_shift;
        const int have = (c + page - 1) >> p.page_shift;
        int32_t* const entry = p.table + (long long)lo * p.max_pages + j;
        int id;
        if (j >= have) {
          id = p.pool[(int)(((long long)head + first + (j - have)) % p.pages)];
          if ((pos & (page - 1)) == 0) *entry = id;
        } else {
          id = *entry;
        }
        if (id >= 0 && id < p.pages) slot = (id << p.page_shift) + (pos & (page - 1));
        else bad = true;
      }
    }
    p.slot_map[t] = slot;
  }
  // The ended requests' pages, one warp per request.
  if (all_back) {
    const int lane = tid % 32, warps = gridDim.x * (PLAN_THREADS / 32);
    for (int r = blockIdx.x * (PLAN_THREADS / 32) + tid / 32; r < p.R; r += warps) {
      const int b = s_back[r];
      if (b < 0) continue;
      const int have = (int)((min(max((long long)s_ctx[r], 0LL), cap) + page - 1) >> p.page_shift);
      for (int j = lane; j < have; j += 32) {
        const long long k = (long long)count + b + j;
        if (k < p.pages) p.pool[(int)(((long long)head + k) % p.pages)] = p.table[(long long)r * p.max_pages + j];
      }
    }
  }
  if (bad) atomicOr(p.status, kDevCheck);
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

struct AppendParams {
  const uint16_t* qkv;
  const int32_t* slot_map;
  uint16_t* q;
  uint16_t* k_cache;
  uint16_t* v_cache;
  long long q_stride;
  int T, n_head, n_kv_head, page_shift;
  int slots;  // pages * page_size
  float eps;
};

__global__ void paged_append_kernel(const AppendParams p) {
  pdl_wait();
  pdl_trigger();
  const int t = blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  if (t >= p.T) return;
  const int heads = p.n_head + 2 * p.n_kv_head;
  const uint2* src = reinterpret_cast<const uint2*>(p.qkv + (long long)t * heads * HD) + lane;
  const int slot = p.slot_map[t];
  const bool kept = slot >= 0 && slot < p.slots;
  const int page = kept ? slot >> p.page_shift : 0, off = slot & ((1 << p.page_shift) - 1);
  for (int h = 0; h < heads; ++h) {
    if (h >= p.n_head && !kept) break;
    uint2 v = src[h * (HD / 4)];
    if (h < p.n_head + p.n_kv_head) {
      const float a = __uint_as_float(v.x << 16), b = __uint_as_float(v.x & 0xFFFF0000u);
      const float c = __uint_as_float(v.y << 16), d = __uint_as_float(v.y & 0xFFFF0000u);
      float ss = a * a + b * b + c * c + d * d;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(FULL, ss, o);
      const float f = rsqrtf(ss * (1.0f / HD) + p.eps);
      v = make_uint2(pack_bf16x2(a * f, b * f), pack_bf16x2(c * f, d * f));
    }
    uint16_t* dst;
    if (h < p.n_head) {
      dst = p.q + t * p.q_stride + h * HD;
    } else {
      const int g = (h - p.n_head) % p.n_kv_head;
      const long long row = (((long long)page * p.n_kv_head + g) << p.page_shift) + off;
      dst = (h < p.n_head + p.n_kv_head ? p.k_cache : p.v_cache) + row * HD;
    }
    reinterpret_cast<uint2*>(dst)[lane] = v;
  }
}

int log2_of(int v) {
  int s = 0;
  while ((1 << s) < v) ++s;
  return s;
}

}  // namespace

cudaError_t launch_paged_plan(const moe_paged_shape_t& s, const int32_t* ctx_len, const int32_t* new_len,
                              int32_t* block_table, int32_t* pool, const int32_t* pool_in, int32_t* pool_out,
                              int32_t* row_start, int32_t* slot_map, int32_t* kv_len, int32_t* next_ctx, int32_t* info,
                              cudaStream_t st) {
  PlanParams p{ctx_len, new_len, block_table, pool, pool_in, pool_out, row_start, slot_map, kv_len, next_ctx, info,
               device_status_ptr(), s.requests, s.tokens, s.pages, s.max_pages, log2_of(s.page_size)};
  if (!p.status) return cudaErrorInvalidDevicePointer;
  const size_t smem = sizeof(int32_t) * (4 * (size_t)s.requests + 1);
  const cudaError_t e = cudaFuncSetAttribute(paged_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)(sizeof(int32_t) * (4 * kPagedMaxRequests + 1)));
  if (e != cudaSuccess) return e;
  const int blocks = (s.tokens + PLAN_THREADS - 1) / PLAN_THREADS;
  return launch_pdl(paged_plan_kernel, dim3((unsigned)(blocks < 152 ? blocks : 152)), dim3(PLAN_THREADS), smem, st, p);
}

cudaError_t launch_paged_append(const moe_paged_shape_t& s, const uint16_t* qkv, const int32_t* slot_map, uint16_t* q,
                                long long q_stride, uint16_t* k_cache, uint16_t* v_cache, cudaStream_t st) {
  const AppendParams p{qkv, slot_map, q, k_cache, v_cache, q_stride, s.tokens, s.n_head, s.n_kv_head,
                       log2_of(s.page_size), s.pages * s.page_size, s.eps};
  return launch_pdl(paged_append_kernel, dim3((unsigned)((s.tokens + 7) / 8)), dim3(256), 0, st, p);
}

}  // namespace moe
