// Causal grouped-query attention of a step's new tokens over a paged key/value cache.
//
// Simple form: one warp per (token row, query head), four of the head's 128 values per
// lane, one pass over the keys with the running maximum and sum of the softmax.
#include <cuda_bf16.h>
#include <math.h>

#include "internal.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr unsigned FULL = 0xFFFFFFFFu;
constexpr int HD = kAttnHeadDim;

struct PagedParams {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  const int32_t* table;
  const int32_t* row_start;
  const int32_t* kv_len;
  uint16_t* out;
  float* lse;
  int* status;
  long long q_stride;
  int R, T, n_head, n_kv_head, pages, max_pages, page_shift;
  float scale;
};

__device__ __forceinline__ float4 load4(const uint16_t* p) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u), __uint_as_float(v.y << 16),
                     __uint_as_float(v.y & 0xFFFF0000u));
}

__global__ void paged_attention_kernel(const PagedParams p) {
  pdl_wait();
  pdl_trigger();
  const long long w = (long long)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  if (w >= (long long)p.T * p.n_head) return;
  const int t = (int)(w / p.n_head), h = (int)(w % p.n_head);
  const int g = h / (p.n_head / p.n_kv_head);
  int keys = 0, r = 0;
  if (t >= p.row_start[0] && t < p.row_start[p.R]) {
    int lo = 0, hi = p.R;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.row_start[mid] <= t) lo = mid;
      else hi = mid;
    }
    r = lo;
    const int n = p.row_start[r + 1] - p.row_start[r];
    const int len = p.kv_len[r];
    if (len >= n) keys = len - n + (t - p.row_start[r]) + 1;
    if (len > (p.max_pages << p.page_shift)) {
      keys = 0;
      if (lane == 0) atomicOr(p.status, kDevCheck);
    }
  }
  const float4 q = load4(p.q + t * p.q_stride + h * HD + lane * 4);
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  const int page = 1 << p.page_shift;
  for (int k = 0; k < keys; ++k) {
    const int id = p.table[(long long)r * p.max_pages + (k >> p.page_shift)];
    if (id < 0 || id >= p.pages) {
      if (lane == 0) atomicOr(p.status, kDevCheck);
      continue;
    }
    const long long row = ((((long long)id * p.n_kv_head + g) << p.page_shift) + (k & (page - 1))) * HD + lane * 4;
    const float4 kk = load4(p.k + row), vv = load4(p.v + row);
    float s = q.x * kk.x + q.y * kk.y + q.z * kk.z + q.w * kk.w;
#pragma unroll
    for (int b = 16; b > 0; b >>= 1) s += __shfl_xor_sync(FULL, s, b);
    s *= p.scale;
    const float mn = fmaxf(m, s), f = expf(m - mn), e = expf(s - mn);
    m = mn;
    l = l * f + e;
    o = make_float4(o.x * f + e * vv.x, o.y * f + e * vv.y, o.z * f + e * vv.z, o.w * f + e * vv.w);
  }
  const float inv = l > 0.f ? 1.0f / l : 0.f;
  const __nv_bfloat162 a = __floats2bfloat162_rn(o.x * inv, o.y * inv), b = __floats2bfloat162_rn(o.z * inv, o.w * inv);
  uint2 packed;
  packed.x = *reinterpret_cast<const uint32_t*>(&a);
  packed.y = *reinterpret_cast<const uint32_t*>(&b);
  *reinterpret_cast<uint2*>(p.out + ((long long)t * p.n_head + h) * HD + lane * 4) = packed;
  if (p.lse && lane == 0) p.lse[(long long)t * p.n_head + h] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace

size_t paged_attention_scratch_bytes(const moe_paged_shape_t&) { return 16; }

cudaError_t launch_paged_attention(const moe_paged_shape_t& s, const uint16_t* q, long long q_stride,
                                   const uint16_t* k_cache, const uint16_t* v_cache, const int32_t* block_table,
                                   const int32_t* row_start, const int32_t* kv_len, uint16_t* out, float* lse, void*,
                                   cudaStream_t st) {
  int shift = 0;
  while ((1 << shift) < s.page_size) ++shift;
  PagedParams p{q, k_cache, v_cache, block_table, row_start, kv_len, out, lse, device_status_ptr(), q_stride,
                s.requests, s.tokens, s.n_head, s.n_kv_head, s.pages, s.max_pages, shift, 1.0f / sqrtf((float)HD)};
  if (!p.status) return cudaErrorInvalidDevicePointer;
  const long long warps = (long long)s.tokens * s.n_head;
  return launch_pdl(paged_attention_kernel, dim3((unsigned)((warps + 7) / 8)), dim3(256), 0, st, p);
}

}  // namespace moe
