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
// token; it is bound by the launch and the chain load - sums - search - pool load - store: 3.2
// to 3.7 us a launch for a step of up to 8 requests, 6.6 us for 1021 requests and 8072 rows (with
// the ctypes call around it 4.9 and 7.2 us; the first form, sums in one serial pass: 9.9 and 11.2).
// In place a step of one CTA costs the same, a larger one a second small launch (paged_advance_kernel).
//
// paged_append_kernel: one warp per token row; q and k heads normalised in fp32, q to its
// row, k and v to their page.  A copy with a reduction, bound by memory traffic: 8192 rows of
// 8 + 2 + 2 heads (50 MB) in 8.4 us among other calls, 7.0 us back to back in a captured graph
// where the writes stay in L2, 12.2 us under ncu with cold caches; 64 rows in 2.8 us.
#include <cuda_bf16.h>

#include <algorithm>

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
  const int32_t* pool_in;  // with one CTA pool_out may be pool_in, next_ctx ctx_len: both are read
  int32_t* pool_out;       // ahead of the first barrier and written behind it.  Null: left to
                           // paged_advance_kernel
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

// The last index r of the non-decreasing v[0 .. n] with v[r] <= x, where v[0] <= x < v[n].
__device__ __forceinline__ int find_range(const int32_t* v, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (v[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(PLAN_THREADS) paged_plan_kernel(const PlanParams p) {
  extern __shared__ int32_t plan_smem[];
  int32_t* const s_ctx = plan_smem;          // [R]
  int32_t* const s_new = s_ctx + p.R;        // [R] new tokens, then the place of the request's first
                                             //     fresh page counted from the pool's head; -1 = denied
  int32_t* const s_row = s_new + p.R;        // [R + 1] row starts, at most T
  int32_t* const s_back = s_row + p.R + 1;   // [R + 1] first returned page, counted from the pool's count
  __shared__ long long warp_sums[PLAN_THREADS / 32];
  const int tid = threadIdx.x;
  const int page = 1 << p.page_shift;
  const long long cap = (long long)p.max_pages << p.page_shift;
  pdl_wait();
  pdl_trigger();
  const int head_in = p.pool_in[0], count_in = p.pool_in[1];
  for (int r = tid; r < p.R; r += PLAN_THREADS) {
    s_ctx[r] = p.ctx_len[r];
    s_new[r] = p.new_len[r];
  }
  const bool pool_ok = head_in >= 0 && head_in < p.pages && count_in >= 0 && count_in <= p.pages;
  const int head = pool_ok ? head_in : 0, count = pool_ok ? count_in : 0;
  bool bad = !pool_ok;
  __syncthreads();

  // This thread's requests: a contiguous run, so that its sums extend the block's.
  const int per = (p.R + PLAN_THREADS - 1) / PLAN_THREADS;
  const int r0 = min(p.R, tid * per), r1 = min(p.R, r0 + per);
  auto held = [&](int c) { return (int)((min(max((long long)c, 0LL), cap) + page - 1) >> p.page_shift); };
  // Pages that a request with n > 0 new tokens, the last of them in row `end_row` - 1, begins; -1: no fit.
  auto wanted = [&](int c, int n, long long end_row) {
    const long long end = (long long)c + n;
    if (c < 0 || end > cap || end_row > p.T) return -1;
    return (int)((end + page - 1) >> p.page_shift) - held(c);
  };
  long long rows = 0;
  for (int r = r0; r < r1; ++r) rows += max(s_new[r], 0);
  long long all_rows, all_need, all_back;
  const long long row0 = block_exclusive_sum(rows, warp_sums, &all_rows);

  long long need = 0, back = 0, row = row0;
  for (int r = r0; r < r1; ++r) {
    const int c = s_ctx[r], n = s_new[r];
    s_row[r] = (int)min(row, (long long)p.T);
    row += max(n, 0);
    if (c < 0 || c > cap) bad = true;
    if (n > 0) {
      const int w = wanted(c, n, row);
      if (w < 0) bad = true;
      need += max(w, 0);
    } else if (n < 0) {
      back += held(c);
    }
  }
  const long long need0 = block_exclusive_sum(need, warp_sums, &all_need);
  const long long back0 = block_exclusive_sum(back, warp_sums, &all_back);

  const bool first_cta = blockIdx.x == 0;
  long long upto = need0, ret = back0, taken = 0, denied = 0;
  row = row0;
  for (int r = r0; r < r1; ++r) {
    const int c = s_ctx[r], n = s_new[r];
    row += max(n, 0);
    s_back[r] = (int)min(ret, (long long)p.pages);
    bool granted = false;
    if (n > 0) {
      const int w = wanted(c, n, row);
      upto += max(w, 0);
      granted = w == 0 || (w > 0 && upto <= count);
      s_new[r] = granted ? (int)(w ? upto - w : 0) : -1;
      if (granted && w) taken = upto;
      if (!granted) ++denied;
    } else if (n < 0) {
      ret += held(c);
    }
    if (first_cta) {
      p.row_start[r] = s_row[r];
      p.kv_len[r] = granted ? c + n : n == 0 ? c : 0;
      if (p.next_ctx) p.next_ctx[r] = granted ? c + n : n < 0 ? 0 : c;
    }
  }
  const int used = (int)min(all_rows, (long long)p.T), returned = (int)min(all_back, (long long)p.pages);
  if (tid == 0) {
    s_row[p.R] = used;
    s_back[p.R] = returned;
  }
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
      // No more than `pages` pages are free: a caller that returns a page twice is told so.
      if (count + all_back > p.pages) bad = true;
      p.row_start[p.R] = used;
      if (p.pool_out) {
        p.pool_out[0] = (int)(((long long)head + s_taken) % p.pages);
        p.pool_out[1] = (int)min(count - s_taken + all_back, (long long)p.pages);
      }
      p.info[0] = used;
      p.info[1] = s_taken;
      p.info[2] = returned;
      p.info[3] = (int)all_denied;
    }
  }
  __syncthreads();

  // The rows' slots; a token at the first position of a page writes its table entry.
  auto ring = [&](int place) {  // place < 2 pages
    const long long x = (long long)head + place;
    return (int)(x >= p.pages ? x - p.pages : x);
  };
  for (int t = blockIdx.x * PLAN_THREADS + tid; t < p.T; t += gridDim.x * PLAN_THREADS) {
    int slot = -1;
    if (t < used) {
      const int r = find_range(s_row, p.R, t), first = s_new[r];
      if (first >= 0) {
        const int c = s_ctx[r], pos = c + (t - s_row[r]), j = pos >> p.page_shift;
        const int have = (c + page - 1) >> p.page_shift;
        int32_t* const entry = p.table + (long long)r * p.max_pages + j;
        int id;
        if (j >= have) {
          id = p.pool[ring(first + (j - have))];
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
  // The ended requests' pages, behind the free ones.
  for (int k = blockIdx.x * PLAN_THREADS + tid; k < returned && count + k < p.pages; k += gridDim.x * PLAN_THREADS) {
    const int r = find_range(s_back, p.R, k);
    const int id = p.table[(long long)r * p.max_pages + (k - s_back[r])];
    if (id < 0 || id >= p.pages) bad = true;
    p.pool[ring(count + k)] = id;
  }
  if (bad) atomicOr(p.status, kDevCheck);
}

// A step in place that several CTAs plan: the contexts and the pool's state are replaced by a
// launch of its own, once every CTA of the plan has read them.  What it needs is among the plan's
// outputs: a request's next context is its kv_len, but 0 if it ended and the present one if it was
// denied (new tokens and no keys).
__global__ void __launch_bounds__(PLAN_THREADS) paged_advance_kernel(int32_t* ctx, const int32_t* new_len,
                                                                     const int32_t* kv_len, int32_t* pool_state,
                                                                     const int32_t* info, int R, int pages) {
  pdl_wait();
  pdl_trigger();
  const int r = blockIdx.x * PLAN_THREADS + threadIdx.x;
  if (ctx && r < R) {
    const int n = new_len[r], kv = kv_len[r];
    if (n < 0) ctx[r] = 0;
    else if (n > 0 && kv > 0) ctx[r] = kv;
  }
  if (pool_state && r == 0) {
    const int head = pool_state[0], count = pool_state[1], taken = info[1], returned = info[2];
    const bool ok = head >= 0 && head < pages && count >= 0 && count <= pages;  // else nothing was taken
    pool_state[0] = ok ? (int)(((long long)head + taken) % pages) : 0;
    pool_state[1] = (int)min((ok ? count - taken : 0) + (long long)returned, (long long)pages);
  }
}

struct AppendParams {
  const uint16_t* qkv;
  const int32_t* slot_map;
  const int32_t* used;  // rows in use: the others have no slot, whatever the map holds there; null = all rows
  uint16_t* q;
  uint16_t* k_cache;
  uint16_t* v_cache;
  long long q_stride;
  int T, n_head, n_kv_head, page_shift;
  int slots;  // pages * page_size
  float eps;
};

// Half a warp per head, 16 bytes per lane; up to sixteen heads' loads are on their way before
// the first reduction.  Bound by the memory system: 8192 rows of 8 + 2 + 2 heads move 50 MB.
constexpr int APPEND_PAIRS = 8;
__global__ void __launch_bounds__(256, 4) paged_append_kernel(const AppendParams p) {
  pdl_wait();
  pdl_trigger();
  const int t = blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32;
  const int lane = threadIdx.x % 32, col = lane & 15, sub = lane >> 4;
  if (t >= p.T) return;
  const int heads = p.n_head + 2 * p.n_kv_head;
  const uint4* src = reinterpret_cast<const uint4*>(p.qkv + (long long)t * heads * HD) + col;
  const int used = p.used ? *p.used : p.T, mapped = p.slot_map[t], slot = t < used ? mapped : -1;
  const bool kept = slot >= 0 && slot < p.slots;
  const int last = kept ? heads : p.n_head;  // a row without a slot has its query heads alone moved
  const long long page = kept ? slot >> p.page_shift : 0;
  const int off = slot & ((1 << p.page_shift) - 1);
  for (int h0 = 0; h0 < last; h0 += 2 * APPEND_PAIRS) {
    uint4 v[APPEND_PAIRS];
#pragma unroll
    for (int i = 0; i < APPEND_PAIRS; ++i) {
      const int h = h0 + 2 * i + sub;
      if (h < last) v[i] = src[h * (HD / 8)];
    }
#pragma unroll
    for (int i = 0; i < APPEND_PAIRS; ++i) {
      const int h = h0 + 2 * i + sub;
      if (h0 + 2 * i >= last) break;
      uint32_t* const w = reinterpret_cast<uint32_t*>(&v[i]);
      float f[8], ss = 0.f;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        f[2 * x] = __uint_as_float(w[x] << 16);
        f[2 * x + 1] = __uint_as_float(w[x] & 0xFFFF0000u);
        ss += f[2 * x] * f[2 * x] + f[2 * x + 1] * f[2 * x + 1];
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(FULL, ss, o);
      if (h >= last) continue;
      if (h < p.n_head + p.n_kv_head) {
        const float r = rsqrtf(ss * (1.0f / HD) + p.eps);
#pragma unroll
        for (int x = 0; x < 4; ++x) w[x] = pack_bf16x2(f[2 * x] * r, f[2 * x + 1] * r);
      }
      uint16_t* dst;
      if (h < p.n_head) {
        dst = p.q + t * p.q_stride + h * HD;
      } else {
        const bool key = h < p.n_head + p.n_kv_head;
        const int g = h - p.n_head - (key ? 0 : p.n_kv_head);
        dst = (key ? p.k_cache : p.v_cache) + (((page * p.n_kv_head + g) << p.page_shift) + off) * HD;
      }
      reinterpret_cast<uint4*>(dst)[col] = v[i];
    }
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
  // Enough threads for the rows, and for an eighth of the tables' pages coming back at once.
  const long long work = std::max<long long>(s.tokens, (long long)s.requests * s.max_pages / 8);
  const long long blocks = std::min<long long>((work + PLAN_THREADS - 1) / PLAN_THREADS, 152);
  int32_t* const ctx_late = blocks > 1 && next_ctx == ctx_len ? next_ctx : nullptr;
  int32_t* const pool_late = blocks > 1 && pool_out == pool_in ? pool_out : nullptr;
  PlanParams p{ctx_len, new_len, block_table, pool, pool_in, pool_late ? nullptr : pool_out, row_start, slot_map,
               kv_len, ctx_late ? nullptr : next_ctx, info, device_status_ptr(), s.requests, s.tokens, s.pages,
               s.max_pages, log2_of(s.page_size)};
  if (!p.status) return cudaErrorInvalidDevicePointer;
  const size_t smem = sizeof(int32_t) * (4 * (size_t)s.requests + 2);
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(paged_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)(sizeof(int32_t) * (4 * kPagedMaxRequests + 2)));
    if (e != cudaSuccess) return e;
  }
  const cudaError_t e = launch_pdl(paged_plan_kernel, dim3((unsigned)blocks), dim3(PLAN_THREADS), smem, st, p);
  if (e != cudaSuccess || (!ctx_late && !pool_late)) return e;
  const unsigned rows = ctx_late ? (unsigned)s.requests : 1u;
  return launch_pdl(paged_advance_kernel, dim3((rows + PLAN_THREADS - 1) / PLAN_THREADS), dim3(PLAN_THREADS), 0, st,
                    ctx_late, new_len, (const int32_t*)kv_len, pool_late, (const int32_t*)info, s.requests, s.pages);
}

cudaError_t launch_paged_append(const moe_paged_shape_t& s, const uint16_t* qkv, const int32_t* slot_map,
                                const int32_t* used, uint16_t* q, long long q_stride, uint16_t* k_cache,
                                uint16_t* v_cache, cudaStream_t st) {
  const AppendParams p{qkv, slot_map, used, q, k_cache, v_cache, q_stride, s.tokens, s.n_head, s.n_kv_head,
                       log2_of(s.page_size), s.pages * s.page_size, s.eps};
  return launch_pdl(paged_append_kernel, dim3((unsigned)((s.tokens + 7) / 8)), dim3(256), 0, st, p);
}

}  // namespace moe
