// QK-norm with rotary positions in one pass (sm_103a): the rows of a serving step with the cache
// write, whole sequences forward, and the backward of that.
//
// Relay article ("Una carrera de relevos con GPUs alquiladas entrenó el MoE de 2.7B de
// NanoColibri por $200"), opening section, architecture paragraph: a per-head QK-norm; the
// article names no positions, so their form is this library's own.
//
// n = u r with r = (mean(u^2) + eps)^-1/2 over a head's 128 values; then every pair (a, b) of the
// head's first rotary_dim values becomes m (a cos t - b sin t, b cos t + a sin t), t the pair's angle.
//
// Angles.  A pair's frequency is a fraction of a turn per token in units of 2^-64 (moe_rope_t), so
// that position times frequency modulo 2^64 is the angle with the whole turns gone, exact at any
// position: one 64-bit integer product whose upper 32 bits, as a signed number, are the angle in
// units of 2^-31 half turns.  In fp32 radians a position of 2^17 would be off by 2^-7, and fp64
// arithmetic runs at a sixty-fourth of the fp32 rate here.  The hardware's sine and cosine of it, once
// per row and pair, both together within 2^-20.7 of the pair's length (the two bounds of the programming guide over
// half a turn either way); with the angle's 32 bits, the norm and the products below 2^-18, where the output's
// rounding is 2^-8 of a value.
//
// Layout.  One warp per row, half a warp per head, sixteen bytes per lane, up to sixteen heads'
// loads on their way before the first reduction.  A lane holds both values of four pairs whatever
// the layout, so that no value crosses lanes: neighbouring pairs lie in its sixteen bytes anyway;
// for halves lane l takes values 4 l .. 4 l + 3 of the first half and of the second.
//
// Sums, norms, angles and products in fp32, one rounding to bf16 at the end.
//
// Bound by memory traffic; back to back in a graph, inputs in L2 and (in brackets) from HBM: append of 8192 rows of
// 8 + 2 + 2 heads (50 MB) 8.3 us (10.9, 4.6 TB/s), of 64 rows 3.0 us, forward and backward of 8192 rows (122 MB) 17.0 us
// (21.6, 5.6 TB/s).  With sincospif, eight rows to a block and the row's place found before its first loads the
// append took 11.0 us (inputs in L2).  A warp that takes several rows and loads the next one ahead: 11.5 for 10.9 us.
// Without a rotation the block's calls keep to the kernels that have none: paged_append_kernel takes 6.9 us where
// this one takes 8.5 (8192 rows; 2.7 and 3.1 for 64 rows, back to back in a graph), and the dense block of 8192 rows the
// same with either norm (99.2 to 99.6 us).
#include <cuda_bf16.h>
#include <math.h>

#include "internal.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr unsigned FULL = 0xFFFFFFFFu;
constexpr int HD = kAttnHeadDim;
constexpr int PAIRS_MAX = HD / 2;
constexpr int ROWS_PER_BLOCK = 4;
constexpr int FWD_BATCH = 6, BWD_BATCH = 3;  // heads per half warp whose loads are on their way together
constexpr float PI = 3.14159265358979f;

struct Rotation {
  uint64_t turns[PAIRS_MAX];
  int lanes;  // rotary_dim / 8: the lanes of a half warp that hold pairs
  float magnitude;
};
Rotation rotation_of(const moe_rope_t* rope) {
  Rotation r{};
  if (!rope) return r;  // no lane turns anything
  for (int i = 0; i < rope->rotary_dim / 2; ++i) r.turns[i] = rope->turns[i];
  r.lanes = rope->rotary_dim / 8;
  r.magnitude = rope->magnitude;
  return r;
}

struct NormRopeParams {
  Rotation rot;
  const uint16_t* qkv;
  uint16_t* out;  // q rows of a serving step, or all heads
  long long out_stride;
  int T, n_head, n_kv_head;
  float eps;
  // whole sequences
  const int32_t* positions;  // null: row % seq
  int seq;
  int heads;  // moved: without the value heads where out is qkv
  // a serving step
  const int32_t* slot_map;
  const int32_t* row_start;
  const int32_t* kv_len;
  uint16_t* k_cache;
  uint16_t* v_cache;
  int R, page_shift, slots;
};

// A lane's eight values of a head: chunks of four at elements a and b.
struct Chunks {
  int a, b;
};
template <bool PAIRS>
__device__ __forceinline__ Chunks chunks_of(int col, int lanes) {
  if (PAIRS || col >= lanes) return {8 * col, 8 * col + 4};
  return {4 * col, 4 * (col + lanes)};
}
struct Vals {
  uint2 a, b;
};
template <bool PAIRS>
__device__ __forceinline__ Vals load_vals(const uint16_t* head, const Chunks& c) {
  if (PAIRS) {
    const uint4 v = *reinterpret_cast<const uint4*>(head + c.a);
    return {make_uint2(v.x, v.y), make_uint2(v.z, v.w)};
  }
  return {*reinterpret_cast<const uint2*>(head + c.a), *reinterpret_cast<const uint2*>(head + c.b)};
}
template <bool PAIRS>
__device__ __forceinline__ void store_vals(uint16_t* head, const Chunks& c, const Vals& v) {
  if (PAIRS) {
    *reinterpret_cast<uint4*>(head + c.a) = make_uint4(v.a.x, v.a.y, v.b.x, v.b.y);
  } else {
    *reinterpret_cast<uint2*>(head + c.a) = v.a;
    *reinterpret_cast<uint2*>(head + c.b) = v.b;
  }
}
// The lane's four pairs as first and second values, two to a register pair: the fp32 pipe's paired
// instructions take both (half as many instructions, which bound these kernels behind the memory).
struct Pairs {
  float2 a[2], b[2];
};
__device__ __forceinline__ float2 lows(uint32_t x, uint32_t y) {
  return make_float2(__uint_as_float(x << 16), __uint_as_float(y << 16));
}
__device__ __forceinline__ float2 highs(uint32_t x, uint32_t y) {
  return make_float2(__uint_as_float(x & 0xFFFF0000u), __uint_as_float(y & 0xFFFF0000u));
}
__device__ __forceinline__ float2 both(uint32_t x) {
  return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u));
}
template <bool PAIRS>
__device__ __forceinline__ Pairs unpack(const Vals& v) {
  if (PAIRS) return {{lows(v.a.x, v.a.y), lows(v.b.x, v.b.y)}, {highs(v.a.x, v.a.y), highs(v.b.x, v.b.y)}};
  return {{both(v.a.x), both(v.a.y)}, {both(v.b.x), both(v.b.y)}};
}
template <bool PAIRS>
__device__ __forceinline__ Vals pack(const Pairs& p) {
  if (PAIRS)
    return {make_uint2(pack_bf16x2(p.a[0].x, p.b[0].x), pack_bf16x2(p.a[0].y, p.b[0].y)),
            make_uint2(pack_bf16x2(p.a[1].x, p.b[1].x), pack_bf16x2(p.a[1].y, p.b[1].y))};
  return {make_uint2(pack_bf16x2(p.a[0].x, p.a[0].y), pack_bf16x2(p.a[1].x, p.a[1].y)),
          make_uint2(pack_bf16x2(p.b[0].x, p.b[0].y), pack_bf16x2(p.b[1].x, p.b[1].y))};
}
__device__ __forceinline__ float dot(const Pairs& x, const Pairs& y) {
  float2 s = __fmul2_rn(x.a[0], y.a[0]);
  s = __ffma2_rn(x.a[1], y.a[1], s);
  s = __ffma2_rn(x.b[0], y.b[0], s);
  s = __ffma2_rn(x.b[1], y.b[1], s);
  return s.x + s.y;
}
__device__ __forceinline__ void scale(Pairs& x, float f) {
  const float2 r = make_float2(f, f);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    x.a[i] = __fmul2_rn(x.a[i], r);
    x.b[i] = __fmul2_rn(x.b[i], r);
  }
}

// The row's rotation, of the lane's four pairs.
struct Turn {
  float2 c[2], s[2];
  bool on;
};
__device__ __forceinline__ Turn turn_of(const uint64_t* turns, const Rotation& rot, int col, int pos) {
  Turn t;
  t.on = col < rot.lanes;
  float c[4], s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t at = (uint64_t)(int64_t)pos * turns[4 * col + i];
    const float half_turns = (float)(int32_t)(at >> 32) * 0x1p-31f;
    c[i] = __cosf(half_turns * PI) * rot.magnitude;
    s[i] = __sinf(half_turns * PI) * rot.magnitude;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    t.c[i] = make_float2(c[2 * i], c[2 * i + 1]);
    t.s[i] = make_float2(s[2 * i], s[2 * i + 1]);
  }
  return t;
}
// BACK: the transposed rotation.
template <bool BACK>
__device__ __forceinline__ void rotate(Pairs& x, const Turn& t) {
  if (!t.on) return;  // what is not turned is not multiplied either: 0 times an infinity is none
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 a = x.a[i], b = x.b[i], up = t.s[i], down = make_float2(-up.x, -up.y);
    x.a[i] = __ffma2_rn(b, BACK ? up : down, __fmul2_rn(a, t.c[i]));
    x.b[i] = __ffma2_rn(a, BACK ? down : up, __fmul2_rn(b, t.c[i]));
  }
}
__device__ __forceinline__ float half_warp_sum(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
  return v;
}

// The position of row t < row_start[R]; all lanes of a warp search its request together, 32 places at a time
// and the last 32 with their lengths at once (up to 32 requests: one round of loads).  What row_start holds
// decides no address outside [0, R].
__device__ __forceinline__ int position_of(const NormRopeParams& p, int t, int lane) {
  int lo = 0, hi = p.R;  // row_start[lo] <= t
  while (hi - lo > 32) {
    const int step = (hi - lo + 31) >> 5, at = lo + (lane + 1) * step;
    const bool below = at < hi && p.row_start[at] <= t;
    lo += __popc(__ballot_sync(FULL, below)) * step;
    hi = min(hi, lo + step);
  }
  const int at = min(lo + lane, p.R - 1);
  const int first = p.row_start[lo], end = p.row_start[at + 1], len = p.kv_len[at];
  const int r = min(__popc(__ballot_sync(FULL, lo + lane < hi && end <= t)), 31);
  const int a = __shfl_sync(FULL, end, max(r - 1, 0)), b = __shfl_sync(FULL, end, r), kv = __shfl_sync(FULL, len, r);
  const int start = r > 0 ? a : first, n = b - start;
  return kv >= n ? kv - n + (t - start) : 0;
}

template <bool PAIRS, bool PAGED>
__global__ void __launch_bounds__(32 * ROWS_PER_BLOCK, 8) norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
  __shared__ uint64_t s_turns[PAIRS_MAX];
  if (threadIdx.x < PAIRS_MAX) s_turns[threadIdx.x] = p.rot.turns[threadIdx.x];
  pdl_wait();
  pdl_trigger();
  __syncthreads();
  const int t = blockIdx.x * ROWS_PER_BLOCK + threadIdx.x / 32;
  const int lane = threadIdx.x % 32, col = lane & 15, sub = lane >> 4;
  if (t >= p.T) return;
  const int heads = p.n_head + 2 * p.n_kv_head;  // PAGED: p.heads
  const uint16_t* const src = p.qkv + (long long)t * heads * HD;
  const Chunks at = chunks_of<PAIRS>(col, p.rot.lanes);
  int last = p.heads, slot = -1;
  Turn turn;
  for (int h0 = 0; h0 < last; h0 += 2 * FWD_BATCH) {
    Vals v[FWD_BATCH];
#pragma unroll
    for (int i = 0; i < FWD_BATCH; ++i) {
      const int h = h0 + 2 * i + sub;
      if (h < (PAGED ? heads : last)) v[i] = load_vals<PAIRS>(src + h * HD, at);
    }
    if (h0 == 0) {  // the row's place and angles, while its first heads are on their way
      int pos;
      if (PAGED) {
        const int used = p.row_start[p.R], mapped = p.slot_map[t];
        pos = position_of(p, t, lane);
        if (t >= used) pos = 0;
        slot = t < used && mapped >= 0 && mapped < p.slots ? mapped : -1;
        last = slot >= 0 ? heads : p.n_head;  // a row without a slot has its query heads alone moved
      } else {
        pos = p.positions ? p.positions[t] : t % p.seq;
      }
      turn = turn_of(s_turns, p.rot, col, pos);
    }
#pragma unroll
    for (int i = 0; i < FWD_BATCH; ++i) {
      const int h = h0 + 2 * i + sub;
      if (h0 + 2 * i >= last) break;
      Pairs x = unpack<PAIRS>(v[i]);
      const float ss = half_warp_sum(dot(x, x));
      if (h >= last) continue;
      if (h < p.n_head + p.n_kv_head) {
        scale(x, rsqrtf(ss * (1.0f / HD) + p.eps));
        rotate<false>(x, turn);
        v[i] = pack<PAIRS>(x);
      }
      uint16_t* dst;
      if (!PAGED || h < p.n_head) {
        dst = p.out + t * p.out_stride + h * HD;
      } else {
        const bool key = h < p.n_head + p.n_kv_head;
        const int g = h - p.n_head - (key ? 0 : p.n_kv_head);
        const long long row = (((long long)(slot >> p.page_shift) * p.n_kv_head + g) << p.page_shift) +
                              (slot & ((1 << p.page_shift) - 1));
        dst = (key ? p.k_cache : p.v_cache) + row * HD;
      }
      store_vals<PAIRS>(dst, at, v[i]);
    }
  }
}

struct NormRopeBwdParams {
  Rotation rot;
  const uint16_t* qkv;
  const uint16_t* dout;
  uint16_t* dqkv;
  const int32_t* positions;
  int T, seq, n_qk, heads;  // query and key heads; heads in a row
  int moved;                // heads to write: without the value heads where dqkv is dout
  float eps;
};

// dn = m R^T dy, du = r (dn - n mean(n dn)).  Both sums of a head go through the same shuffles;
// the norm is computed again from the rows instead of being kept by the forward: its input is
// read for n anyway.  Bound by memory traffic.
template <bool PAIRS>
__global__ void __launch_bounds__(32 * ROWS_PER_BLOCK, 8)
    norm_rope_bwd_kernel(const __grid_constant__ NormRopeBwdParams p) {
  __shared__ uint64_t s_turns[PAIRS_MAX];
  if (threadIdx.x < PAIRS_MAX) s_turns[threadIdx.x] = p.rot.turns[threadIdx.x];
  pdl_wait();
  pdl_trigger();
  __syncthreads();
  const int t = blockIdx.x * ROWS_PER_BLOCK + threadIdx.x / 32;
  const int lane = threadIdx.x % 32, col = lane & 15, sub = lane >> 4;
  if (t >= p.T) return;
  const long long row = (long long)t * p.heads * HD;
  const Chunks at = chunks_of<PAIRS>(col, p.rot.lanes);
  Turn turn;
  for (int h0 = 0; h0 < p.moved; h0 += 2 * BWD_BATCH) {
    Vals u[BWD_BATCH], g[BWD_BATCH];
#pragma unroll
    for (int i = 0; i < BWD_BATCH; ++i) {
      const int h = h0 + 2 * i + sub;
      if (h < p.moved) g[i] = load_vals<PAIRS>(p.dout + row + h * HD, at);
      if (h < p.n_qk) u[i] = load_vals<PAIRS>(p.qkv + row + h * HD, at);
    }
    if (h0 == 0) turn = turn_of(s_turns, p.rot, col, p.positions ? p.positions[t] : t % p.seq);
#pragma unroll
    for (int i = 0; i < BWD_BATCH; ++i) {
      const int h = h0 + 2 * i + sub;
      if (h0 + 2 * i >= p.moved) break;
      const Pairs f = unpack<PAIRS>(u[i]);
      Pairs d = unpack<PAIRS>(g[i]);
      rotate<true>(d, turn);
      const float ss = half_warp_sum(dot(f, f)), fd = half_warp_sum(dot(f, d));
      if (h >= p.moved) continue;
      if (h < p.n_qk) {
        const float r = rsqrtf(ss * (1.0f / HD) + p.eps);
        const float k = -fd * r * (1.0f / HD) * r;  // - mean(n dn) r: n = u r
        const float2 kk = make_float2(k, k);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          d.a[x] = __ffma2_rn(f.a[x], kk, d.a[x]);
          d.b[x] = __ffma2_rn(f.b[x], kk, d.b[x]);
        }
        scale(d, r);
        g[i] = pack<PAIRS>(d);
      }
      store_vals<PAIRS>(p.dqkv + row + h * HD, at, g[i]);
    }
  }
}

dim3 grid_of(int rows) { return dim3((unsigned)((rows + ROWS_PER_BLOCK - 1) / ROWS_PER_BLOCK)); }
bool pairs_of(const moe_rope_t* rope) { return !rope || rope->layout == MOE_ROPE_INTERLEAVED; }

}  // namespace

moe_status_t check_rope(const moe_rope_t* rope) {
  if (!rope) return MOE_OK;
  if (rope->rotary_dim < 16 || rope->rotary_dim > HD || rope->rotary_dim % 16) return MOE_ERR_UNSUPPORTED;
  if (rope->layout != MOE_ROPE_HALVES && rope->layout != MOE_ROPE_INTERLEAVED) return MOE_ERR_INVALID_ARG;
  if (!(rope->magnitude > 0.f) || !isfinite(rope->magnitude)) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

cudaError_t launch_norm_rope(const moe_attn_shape_t& s, const moe_rope_t* rope, const int32_t* positions,
                             const uint16_t* qkv, uint16_t* out, cudaStream_t st) {
  NormRopeParams p{};
  p.rot = rotation_of(rope);
  p.qkv = qkv;
  p.out = out;
  p.T = s.batch * s.seq;
  p.n_head = s.n_head;
  p.n_kv_head = s.n_kv_head;
  p.out_stride = (long long)(s.n_head + 2 * s.n_kv_head) * HD;
  p.heads = s.n_head + (out == qkv ? 1 : 2) * s.n_kv_head;
  p.eps = s.eps;
  p.positions = positions;
  p.seq = s.seq;
  return launch_pdl(pairs_of(rope) ? norm_rope_kernel<true, false> : norm_rope_kernel<false, false>, grid_of(p.T),
                    dim3(32 * ROWS_PER_BLOCK), 0, st, p);
}

cudaError_t launch_norm_rope_bwd(const moe_attn_shape_t& s, const moe_rope_t* rope, const int32_t* positions,
                                 const uint16_t* qkv, const uint16_t* dout, uint16_t* dqkv, cudaStream_t st) {
  NormRopeBwdParams p{};
  p.rot = rotation_of(rope);
  p.qkv = qkv;
  p.dout = dout;
  p.dqkv = dqkv;
  p.positions = positions;
  p.T = s.batch * s.seq;
  p.seq = s.seq;
  p.n_qk = s.n_head + s.n_kv_head;
  p.heads = s.n_head + 2 * s.n_kv_head;
  p.moved = dqkv == dout ? p.n_qk : p.heads;
  p.eps = s.eps;
  return launch_pdl(pairs_of(rope) ? norm_rope_bwd_kernel<true> : norm_rope_bwd_kernel<false>, grid_of(p.T),
                    dim3(32 * ROWS_PER_BLOCK), 0, st, p);
}

cudaError_t launch_paged_append_rope(const moe_paged_shape_t& s, const moe_rope_t* rope, const uint16_t* qkv,
                                     const int32_t* slot_map, const int32_t* row_start, const int32_t* kv_len,
                                     uint16_t* q, long long q_stride, uint16_t* k_cache, uint16_t* v_cache,
                                     cudaStream_t st) {
  NormRopeParams p{};
  p.rot = rotation_of(rope);
  p.qkv = qkv;
  p.out = q;
  p.out_stride = q_stride;
  p.T = s.tokens;
  p.n_head = s.n_head;
  p.n_kv_head = s.n_kv_head;
  p.heads = s.n_head + 2 * s.n_kv_head;
  p.eps = s.eps;
  p.slot_map = slot_map;
  p.row_start = row_start;
  p.kv_len = kv_len;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.R = s.requests;
  while ((1 << p.page_shift) < s.page_size) ++p.page_shift;
  p.slots = s.pages * s.page_size;
  return launch_pdl(pairs_of(rope) ? norm_rope_kernel<true, true> : norm_rope_kernel<false, true>, grid_of(p.T),
                    dim3(32 * ROWS_PER_BLOCK), 0, st, p);
}

}  // namespace moe

extern "C" moe_status_t moe_rope_init(moe_rope_t* rope, int32_t rotary_dim, int32_t layout, double base, double factor,
                                      int32_t trained_len, double slow_turns, double fast_turns, float magnitude) {
  if (!rope || !(base >= 1.0) || !isfinite(base) || !(factor >= 1.0) || !isfinite(factor) || trained_len < 0)
    return MOE_ERR_INVALID_ARG;
  if (trained_len > 0 && (!(slow_turns >= 0.0) || !(fast_turns > slow_turns) || !isfinite(fast_turns)))
    return MOE_ERR_INVALID_ARG;
  moe_rope_t r{};
  r.rotary_dim = rotary_dim;
  r.layout = layout;
  r.magnitude = magnitude;
  const moe_status_t st = moe::check_rope(&r);
  if (st) return st;
  constexpr double PER_TURN = 0.15915494309189533577;  // 1 / (2 pi)
  for (int i = 0; i < rotary_dim / 2; ++i) {
    double turns = pow(base, -2.0 * i / rotary_dim) * PER_TURN;  // per token
    double kept = 0.0;
    if (trained_len > 0) {
      kept = (trained_len * turns - slow_turns) / (fast_turns - slow_turns);
      kept = kept < 0.0 ? 0.0 : kept > 1.0 ? 1.0 : kept;
    }
    turns *= kept + (1.0 - kept) / factor;
    r.turns[i] = (uint64_t)ldexp(turns, 64);
  }
  *rope = r;
  return MOE_OK;
}
