// C ABI of the paged key/value cache: argument validation, workspace layout and the launch
// sequence of each call.  Declarations and their contracts: moe_gb300.h.
#include <cuda_runtime.h>

#include "internal.h"
#include "moe_gb300.h"

using namespace moe;

namespace {

constexpr size_t kAlign = 1024;
size_t align_up(size_t n) { return (n + kAlign - 1) / kAlign * kAlign; }

bool ok16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

moe_status_t check_paged(const moe_paged_shape_t* s) {
  if (!s) return MOE_ERR_INVALID_ARG;
  if (s->requests < 1 || s->tokens < 1 || s->n_head < 1 || s->n_kv_head < 1 || s->page_size < 1 || s->pages < 1 ||
      s->max_pages < 1 || s->q_stride < 0 || !(s->eps > 0.f))
    return MOE_ERR_INVALID_ARG;
  if (s->q_stride && (s->q_stride % 8 || (long long)s->q_stride < (long long)s->n_head * kAttnHeadDim))
    return MOE_ERR_INVALID_ARG;
  if (s->requests > kPagedMaxRequests || s->tokens > (1 << 20) || s->head_dim != kAttnHeadDim ||
      s->n_head % s->n_kv_head || s->n_head > 8192 / kAttnHeadDim)
    return MOE_ERR_UNSUPPORTED;
  if (s->page_size != 16 && s->page_size != 32 && s->page_size != 64 && s->page_size != 128)
    return MOE_ERR_UNSUPPORTED;
  if ((long long)s->pages * s->n_kv_head * s->page_size >= (1LL << 31) ||
      (long long)s->max_pages * s->page_size > (1LL << 24))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

long long q_stride_of(const moe_paged_shape_t* s) {
  return s->q_stride ? s->q_stride : (long long)s->n_head * kAttnHeadDim;
}

moe_status_t status_of(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

moe_status_t check_block(const moe_paged_shape_t* s, int32_t d) {
  const moe_status_t st = check_paged(s);
  if (st) return st;
  if (d < 1) return MOE_ERR_INVALID_ARG;
  return d % 64 || d > 8192 ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

// The block's workspace: the projected rows, the attention output, the attention's scratch.
struct BlockWs {
  size_t qkv, o, scratch, bytes;
};
BlockWs block_ws(const moe_paged_shape_t* s, int32_t d) {
  const size_t T = (size_t)s->tokens, C = (size_t)(s->n_head + 2 * s->n_kv_head) * kAttnHeadDim;
  BlockWs w;
  w.qkv = 0;
  // The residual path puts the output projection there once q, k and v are done with.
  w.o = align_up(2 * T * (C > (size_t)d ? C : (size_t)d));
  w.scratch = w.o + align_up(2 * T * (size_t)s->n_head * kAttnHeadDim);
  w.bytes = w.scratch + paged_attention_scratch_bytes(*s);
  return w;
}

}  // namespace

extern "C" {

moe_status_t moe_paged_plan(const moe_paged_shape_t* shape, const int32_t* ctx_len, const int32_t* new_len,
                            int32_t* block_table, int32_t* pool, const int32_t* pool_state_in,
                            int32_t* pool_state_out, int32_t* row_start, int32_t* slot_map, int32_t* kv_len,
                            int32_t* next_ctx, int32_t* info, void* stream) {
  const moe_status_t st = check_paged(shape);
  if (st) return st;
  for (const void* p : {(const void*)ctx_len, (const void*)new_len, (const void*)block_table, (const void*)pool,
                        (const void*)pool_state_in, (const void*)pool_state_out, (const void*)row_start,
                        (const void*)slot_map, (const void*)kv_len, (const void*)next_ctx, (const void*)info})
    if (!ok16(p)) return MOE_ERR_INVALID_ARG;
  return status_of(launch_paged_plan(*shape, ctx_len, new_len, block_table, pool, pool_state_in, pool_state_out,
                                     row_start, slot_map, kv_len, next_ctx, info, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_paged_append(const moe_paged_shape_t* shape, const void* qkv, const int32_t* slot_map, void* q,
                              void* k_cache, void* v_cache, void* stream) {
  const moe_status_t st = check_paged(shape);
  if (st) return st;
  if (!ok16(qkv) || !ok16(slot_map) || !ok16(q) || !ok16(k_cache) || !ok16(v_cache)) return MOE_ERR_INVALID_ARG;
  // In place the rows have to be the projection's own.
  if (q == qkv && q_stride_of(shape) != (long long)(shape->n_head + 2 * shape->n_kv_head) * kAttnHeadDim)
    return MOE_ERR_INVALID_ARG;
  return status_of(launch_paged_append(*shape, static_cast<const uint16_t*>(qkv), slot_map, nullptr,
                                       static_cast<uint16_t*>(q), q_stride_of(shape),
                                       static_cast<uint16_t*>(k_cache), static_cast<uint16_t*>(v_cache),
                                       static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_paged_append_rope(const moe_paged_shape_t* shape, const moe_rope_t* rope, const void* qkv,
                                   const int32_t* slot_map, const int32_t* row_start, const int32_t* kv_len, void* q,
                                   void* k_cache, void* v_cache, void* stream) {
  moe_status_t st = check_paged(shape);
  if (!st) st = check_rope(rope);
  if (st) return st;
  if (!ok16(qkv) || !ok16(slot_map) || !ok16(row_start) || !ok16(kv_len) || !ok16(q) || !ok16(k_cache) ||
      !ok16(v_cache))
    return MOE_ERR_INVALID_ARG;
  if (q == qkv && q_stride_of(shape) != (long long)(shape->n_head + 2 * shape->n_kv_head) * kAttnHeadDim)
    return MOE_ERR_INVALID_ARG;
  return status_of(launch_paged_append_rope(*shape, rope, static_cast<const uint16_t*>(qkv), slot_map, row_start,
                                            kv_len, static_cast<uint16_t*>(q), q_stride_of(shape),
                                            static_cast<uint16_t*>(k_cache), static_cast<uint16_t*>(v_cache),
                                            static_cast<cudaStream_t>(stream)));
}

size_t moe_paged_attention_workspace_size(const moe_paged_shape_t* shape) {
  return check_paged(shape) ? 0 : paged_attention_scratch_bytes(*shape);
}

moe_status_t moe_paged_window_attention(const moe_paged_shape_t* shape, int32_t window, int32_t sinks, const void* q,
                                        const void* k_cache, const void* v_cache, const int32_t* block_table,
                                        const int32_t* row_start, const int32_t* kv_len, void* out, float* lse,
                                        void* workspace, size_t ws_bytes, void* stream) {
  const moe_status_t st = check_paged(shape);
  if (st) return st;
  if (window < 0 || sinks < 0) return MOE_ERR_INVALID_ARG;
  if (!ok16(q) || !ok16(k_cache) || !ok16(v_cache) || !ok16(block_table) || !ok16(row_start) || !ok16(kv_len) ||
      !ok16(out) || !ok16(workspace) || (lse && !ok16(lse)))
    return MOE_ERR_INVALID_ARG;
  if (ws_bytes < paged_attention_scratch_bytes(*shape)) return MOE_ERR_WORKSPACE;
  return status_of(launch_paged_window_attention(
      *shape, window, sinks, static_cast<const uint16_t*>(q), q_stride_of(shape),
      static_cast<const uint16_t*>(k_cache), static_cast<const uint16_t*>(v_cache), block_table, row_start, kv_len,
      static_cast<uint16_t*>(out), lse, workspace, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_paged_attention(const moe_paged_shape_t* shape, const void* q, const void* k_cache,
                                 const void* v_cache, const int32_t* block_table, const int32_t* row_start,
                                 const int32_t* kv_len, void* out, float* lse, void* workspace, size_t ws_bytes,
                                 void* stream) {
  return moe_paged_window_attention(shape, 0, 0, q, k_cache, v_cache, block_table, row_start, kv_len, out, lse,
                                    workspace, ws_bytes, stream);
}

size_t moe_attention_paged_workspace_size(const moe_paged_shape_t* shape, int32_t d) {
  return check_block(shape, d) ? 0 : block_ws(shape, d).bytes;
}

moe_status_t moe_attention_paged_window_fwd(const moe_paged_shape_t* shape, int32_t d, const moe_rope_t* rope,
                                            int32_t window, int32_t sinks, const void* x, const void* w_qkv,
                                            const void* w_o, int32_t residual, void* k_cache, void* v_cache,
                                            const int32_t* block_table, const int32_t* row_start,
                                            const int32_t* slot_map, const int32_t* kv_len, void* out, void* workspace,
                                            size_t ws_bytes, void* stream) {
  moe_status_t st = check_block(shape, d);
  if (!st) st = check_rope(rope);
  if (st) return st;
  if (window < 0 || sinks < 0) return MOE_ERR_INVALID_ARG;
  for (const void* p : {x, w_qkv, w_o, (const void*)k_cache, (const void*)v_cache, (const void*)block_table,
                        (const void*)row_start, (const void*)slot_map, (const void*)kv_len, (const void*)out,
                        (const void*)workspace})
    if (!ok16(p)) return MOE_ERR_INVALID_ARG;
  const BlockWs w = block_ws(shape, d);
  if (ws_bytes < w.bytes) return MOE_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* const base = static_cast<uint8_t*>(workspace);
  uint16_t* const qkv = reinterpret_cast<uint16_t*>(base + w.qkv);
  uint16_t* const o = reinterpret_cast<uint16_t*>(base + w.o);
  const int T = shape->tokens, C = (shape->n_head + 2 * shape->n_kv_head) * kAttnHeadDim;
  const int HO = shape->n_head * kAttnHeadDim;
  int bad = 0;
  const CombineInputs none{};
  const GemmOperandSet off{};
  const GemmOperandSet proj{x, T, w_qkv, 1, C, d, qkv, C, EPI_STORE, T};
  cudaError_t e = launch_grouped_gemm(off, nullptr, 1, proj, none, 0, s, &bad);
  if (bad) return MOE_ERR_UNSUPPORTED;
  // The query heads are normalised where the projection left them.  Rows past the plan's write
  // no cache: a slot map that a larger step has filled holds live slots there.  Without a rotation the kernel
  // without one is the faster (rope.cu has the figures).
  if (e == cudaSuccess)
    e = rope ? launch_paged_append_rope(*shape, rope, qkv, slot_map, row_start, kv_len, qkv, C,
                                        static_cast<uint16_t*>(k_cache), static_cast<uint16_t*>(v_cache), s)
             : launch_paged_append(*shape, qkv, slot_map, row_start + shape->requests, qkv, C,
                                   static_cast<uint16_t*>(k_cache), static_cast<uint16_t*>(v_cache), s);
  if (e == cudaSuccess)
    e = launch_paged_window_attention(*shape, window, sinks, qkv, C, static_cast<const uint16_t*>(k_cache),
                                      static_cast<const uint16_t*>(v_cache), block_table, row_start, kv_len, o,
                                      nullptr, base + w.scratch, s);
  if (e != cudaSuccess) return MOE_ERR_CUDA;
  uint16_t* proj_out = residual ? qkv : static_cast<uint16_t*>(out);
  const GemmOperandSet oproj{o, T, w_o, 1, d, HO, proj_out, d, EPI_STORE, T};
  e = launch_grouped_gemm(off, nullptr, 1, oproj, none, 0, s, &bad);
  if (bad) return MOE_ERR_UNSUPPORTED;
  if (e == cudaSuccess && residual)
    e = launch_combine(nullptr, proj_out, nullptr, nullptr, static_cast<const uint16_t*>(x),
                       static_cast<uint16_t*>(out), T, 0, d, s);
  return status_of(e);
}

moe_status_t moe_attention_paged_fwd(const moe_paged_shape_t* shape, int32_t d, const void* x, const void* w_qkv,
                                     const void* w_o, int32_t residual, void* k_cache, void* v_cache,
                                     const int32_t* block_table, const int32_t* row_start, const int32_t* slot_map,
                                     const int32_t* kv_len, void* out, void* workspace, size_t ws_bytes,
                                     void* stream) {
  return moe_attention_paged_window_fwd(shape, d, nullptr, 0, 0, x, w_qkv, w_o, residual, k_cache, v_cache,
                                        block_table, row_start, slot_map, kv_len, out, workspace, ws_bytes, stream);
}

size_t moe_paged_pages_workspace_size(const moe_paged_shape_t* shape) {
  return check_paged(shape) ? 0 : paged_pages_scratch_bytes(*shape);
}

moe_status_t moe_paged_fork(const moe_paged_shape_t* shape, const int32_t* parent, const int32_t* keep, int32_t window,
                            int32_t sinks, const int32_t* ctx_len, const int32_t* table_in, int32_t* table_out,
                            int32_t* pool, const int32_t* pool_state_in, int32_t* pool_state_out, int32_t* next_ctx,
                            int32_t* copies, int32_t* info, void* workspace, size_t ws_bytes, void* stream) {
  const moe_status_t st = check_paged(shape);
  if (st) return st;
  for (const void* p : {(const void*)ctx_len, (const void*)table_in, (const void*)table_out, (const void*)pool,
                        (const void*)pool_state_in, (const void*)pool_state_out, (const void*)next_ctx,
                        (const void*)copies, (const void*)info, (const void*)workspace})
    if (!ok16(p)) return MOE_ERR_INVALID_ARG;
  if ((parent && !ok16(parent)) || (keep && !ok16(keep)) || window < 0 || sinks < 0) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < paged_pages_scratch_bytes(*shape)) return MOE_ERR_WORKSPACE;
  PagesArgs a{};
  a.parent = parent;
  a.keep = keep;
  a.window = window;
  a.sinks = sinks;
  a.ctx_len = ctx_len;
  a.table_in = table_in;
  a.table_out = table_out;
  a.pool = pool;
  a.pool_in = pool_state_in;
  a.pool_out = pool_state_out;
  a.next_ctx = next_ctx;
  a.copies = copies;
  a.info = info;
  return status_of(launch_paged_fork(*shape, a, workspace, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_paged_release(const moe_paged_shape_t* shape, const int32_t* new_len, int32_t window, int32_t sinks,
                               int32_t* ctx_len, int32_t* block_table, int32_t* pool, int32_t* pool_state,
                               int32_t* info, void* workspace, size_t ws_bytes, void* stream) {
  const moe_status_t st = check_paged(shape);
  if (st) return st;
  for (const void* p : {(const void*)new_len, (const void*)ctx_len, (const void*)block_table, (const void*)pool,
                        (const void*)pool_state, (const void*)info, (const void*)workspace})
    if (!ok16(p)) return MOE_ERR_INVALID_ARG;
  if (window < 0 || sinks < 0) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < paged_pages_scratch_bytes(*shape)) return MOE_ERR_WORKSPACE;
  PagesArgs a{};
  a.new_len = new_len;
  a.window = window;
  a.sinks = sinks;
  a.ctx_len = ctx_len;
  a.table_in = block_table;
  a.table_out = block_table;
  a.pool = pool;
  a.pool_in = pool_state;
  a.pool_out = pool_state;
  a.next_ctx = ctx_len;
  a.info = info;
  return status_of(launch_paged_fork(*shape, a, workspace, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_paged_compact(const moe_paged_shape_t* shape, const int32_t* ctx_len, const int32_t* table_in,
                               int32_t* table_out, int32_t* pool, int32_t* pool_state_out, int32_t* copies,
                               int32_t* info, void* workspace, size_t ws_bytes, void* stream) {
  const moe_status_t st = check_paged(shape);
  if (st) return st;
  for (const void* p : {(const void*)ctx_len, (const void*)table_in, (const void*)table_out, (const void*)pool,
                        (const void*)pool_state_out, (const void*)copies, (const void*)info, (const void*)workspace})
    if (!ok16(p)) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < paged_pages_scratch_bytes(*shape)) return MOE_ERR_WORKSPACE;
  PagesArgs a{};
  a.ctx_len = ctx_len;
  a.table_in = table_in;
  a.table_out = table_out;
  a.pool = pool;
  a.pool_out = pool_state_out;
  a.copies = copies;
  a.info = info;
  return status_of(launch_paged_compact(*shape, a, workspace, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_paged_copy(const moe_paged_shape_t* shape, const int32_t* copies, const int32_t* n_copies,
                            int32_t max_copies, int32_t n_caches, void* const* caches, void* stream) {
  const moe_status_t st = check_paged(shape);
  if (st) return st;
  if (!ok16(copies) || !ok16(n_copies) || max_copies < 0 || n_caches < 0 || (n_caches && !caches))
    return MOE_ERR_INVALID_ARG;
  for (int i = 0; i < n_caches; ++i)
    if (!ok16(caches[i])) return MOE_ERR_INVALID_ARG;
  return status_of(launch_paged_copy(*shape, copies, n_copies, max_copies, n_caches, caches,
                                     static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
