// Causal grouped-query attention of a step's new tokens over a paged key/value cache, on
// tcgen05 tensor cores (sm_103a).
//
// Relay article ("Una carrera de relevos con GPUs alquiladas entrenó el MoE de 2.7B de
// NanoColibri por $200"), opening section, architecture paragraph: grouped-query attention;
// the paged cache is this library's own form.
//
// Rows.  The query heads of one key/value head see the same keys, so a tile of queries packs
// them: row m of a 128-row half tile is token m / G, head m % G of the group (G query heads
// per key/value head, tq = 128 / (G rounded up to a power of two) tokens).  One decode token
// fills G rows, a chunk fills all of them, and every key tile is loaded once per group.  A
// work tile is two halves (2 tq tokens): with tokens in both ("pair") the halves share the key
// and value tiles and keep the tensor cores busy in turn; with tokens in the first half only
// ("single") one half's score buffers alternate between key tiles.
//
// Work.  The unit is one 128-key tile of one work tile.  All units of the call, in order
// (request, key/value head, query tile, key tile), are split into equal contiguous ranges, one
// per CTA, whatever the requests' lengths (a work tile counts one unit more than it has key
// tiles, a pair two, for its start and its output): a range holds the end of one work tile,
// whole work tiles and the beginning of another.  A work tile that does not lie in one range
// leaves partial outputs.  A pair's first part is the last work of its range and the others the
// first work of theirs, written long since: with one or two of them the CTA of the first part
// adds them to its own sums.  Other joins (few rows, or many parts) are paged_combine_kernel's,
// eight blocks to a tile.  Either way the order depends on the lengths alone.  Every CTA computes
// the ranges itself from the lengths (one prefix sum over the requests), so the call needs no
// plan, no counters and no cleared workspace.  Rows that belong to no request are the rows of one
// more request without keys; their units read nothing and give zeros.
//
// paged_attention_kernel, one CTA per SM, 18 warps:
//   - warp 16 walks the CTA's range, publishes each item (work tile, key tiles) in a small
//     ring, and issues the TMA copies: the query halves, and one box per page of the key and
//     value tiles, into a ring of five 32 KB stages;
//   - warp 17 (one thread) issues tcgen05.mma: S = Q K^T into a score buffer, O += P V with P
//     (bf16) read from the score buffer's own columns.  The pipe runs in order, so a score
//     product that overwrites a buffer needs no wait for the product that read P from it.  A
//     pair's P comes in three parts (keys 64-127, 0-31, 32-63): the value product of a part runs
//     while the next is computed, and only the last one's lies between the softmax and the next
//     scores (one part: 138 us, two: 129, three: 127 for 2 x 2011 tokens over long contexts, one after
//     the other on one GPU);
//   - warps 0-7 and 8-15, a warp per 16 rows: the online softmax in the log2 domain.  TMEM is
//     read in the 16 x 256-bit shape, four lanes per row with 32 scores each, so that two
//     warps per SM sub-partition share a half tile and the row maximum is two shuffles; O is
//     rescaled only when a row's maximum grew by more than 8 (2^8); at the end O / l, or O, m
//     and l as a partial.  The weights are rounded to bf16, the tensor cores' type beside bf16
//     values; scores, maxima, sums and O stay in fp32, and so do the partials.
// A key that a row does not see has weight 0, but 0 times a NaN or an infinity is not 0.  Values
// past the last key of a work tile are therefore zeroed in shared memory before P V; those that
// its later rows see and its first row does not (as many keys as the tile has tokens, less one) are
// looked through, and a NaN or an infinity among them is taken out and added, at the end, to the
// rows that see it.  Both while the tile's scores are computed, so that it costs little: without
// and with the search four 2048-token prompts took 44.05 and 44.15 us, 13 x 5 tokens 15.2 and 15.7,
// one token over 2047 keys 11.8 and 11.9, over 131070 33.4 and 34.2 (each instruction that a launch
// reaches is fetched anew, so the loops stay rolled: all unrolled 16.0, 12.1 and 34.2; the search
// rolled whole, one 16-byte chunk a turn, takes the prompts to 45.1).
// Every wait for a copy, a product or another CTA is bounded; on a timeout the status word is set
// and the CTA exits.  The issuer's waits for the parts of P are hardware barriers without a limit:
// a half that has an item arrives at every one of them, whatever became of its own waits.
//
// Bounds and measurements (8 query heads on 2 key/value heads; time of a call among others).
// One token for each of 64 requests with 1000 to 16000 keys: 549 MB of keys and values, 93.6 to
// 94.0 us, 5.9 TB/s; between its first copy and its last output a CTA streams at 6.3 TB/s, the
// rest is the start (6 us: two dependent loads, the first copies and each instruction's first
// fetch) and the joins (5 us).  2 x 2011 tokens over 1000 to 14000 keys: 176 GFLOP, 125 to 132 us
// from GPU to GPU (most 130: 1.35 PFLOP/s, 72% of the measured bf16 peak): a half tile's chain
// (3.1k cycles: 0.75k maximum, 1.0k weights, 1.3k from the last part of P over its value product
// and the next scores back to the warps) is longer than both halves' products (2k), and tensor
// memory has no columns for a third half.  Both limits are latency; neither memory nor the pipe
// is saturated.
#include <cuda_bf16.h>
#include <math.h>

#include <atomic>
#include <chrono>
#include <cstddef>
#include <cstring>

#include "internal.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int HD = kAttnHeadDim;
constexpr int BK = 128;                       // keys per tile
constexpr int ATOM_BYTES = 128 * 64 * 2;      // 16 KB: 128 rows x 64 bf16, 128-byte swizzle
constexpr int TILE_BYTES = 2 * ATOM_BYTES;    // 32 KB: 128 rows x 128
constexpr int STAGES = 5;                     // key and value tiles in flight: K0 V0 K1 V1 ...
constexpr int RING_OFF = 2 * TILE_BYTES;      // after the two query halves
constexpr int STATE_OFF = RING_OFF + STAGES * TILE_BYTES;
constexpr int SMEM_BYTES = STATE_OFF + 3072;
constexpr int SOFTMAX_WARPS = 16;             // eight per query half, 16 rows each
constexpr int LOAD_WARP = 16, MMA_WARP = 17;
constexpr int THREADS = 576;
constexpr int WARPS = THREADS / 32;
constexpr int ITEMS = 4;                      // depth of the item ring
constexpr int CTAS = 152;                     // one per SM
constexpr int PART_BAR = 3;                    // hardware barriers 3 .. 8: P's three parts, each of the two halves
constexpr uint32_t O_COL = 256;               // score buffers at 0 and 128, outputs at 256 and 384
constexpr uint32_t TMEM_COLS = 512;
constexpr unsigned FULL = 0xFFFFFFFFu;
constexpr float LN2 = 0.6931471805599453f;

// Partials: per CTA two slots (a work tile continued from the range before; one that goes on in
// the next range), each O [16][256][8] fp32 (groups of eight columns, rows: what a warp stores
// at once is contiguous) and m, l [256].
constexpr size_t PART_O = 16 * 256 * 32;
constexpr size_t PART_BYTES = PART_O + 2 * 256 * 4;

// A part that another CTA adds has a flag per warp that writes it, the call's id once it is
// written; who adds it clears the flag.  Any other value means not written, so the workspace
// needs no clearing.
constexpr int MOST_ADDED = 2;
constexpr size_t FLAG_BYTES = CTAS * SOFTMAX_WARPS * sizeof(unsigned long long);
// A work tile that paged_combine_kernel joins, by the CTA that begins it.
struct Split {
  int row0, ntok, g, last;  // first token row, tokens, key/value head, last CTA with a part (-1: none)
};
constexpr size_t SCRATCH_BYTES = FLAG_BYTES + CTAS * sizeof(Split) + 2 * CTAS * PART_BYTES;

struct PagedParams {
  CUtensorMap q;  // [T] rows viewed as (64, 2, n_head, T), box (64, 1, G, tq)
  CUtensorMap k;  // cache viewed as (64, 8, 2, rows / 8): groups of eight rows, their two column halves; box a page
  CUtensorMap v;
  const int32_t* table;
  const int32_t* row_start;
  const int32_t* kv_len;
  uint16_t* out;
  float* lse;
  unsigned long long* flags;  // [CTA][softmax warp]
  unsigned long long call;    // this call's id
  Split* splits;
  uint8_t* parts;
  int* status;
  int R, T, n_head, n_kv_head, G, tq, tQ_shift, pages, max_pages, page_shift;
  float scale_log2;  // log2(e) / sqrt(HD)
};

struct Item {
  int row0, ntok;   // first token row and tokens of the work tile
  int pos0;         // position of its first token
  int kvlim;        // keys that its last token sees; 0 = a request without keys
  int j0, nt;       // first key tile, key tiles of this item; nt == 0 ends the walk
  int g, half;      // key/value head; query half of a single tile, 2 = pair
  int part;         // partial slot to write; -1 = none: the whole work tile, or the part that adds the others
  int added;        // parts that the first CTA adds to its own; 0 = none
  int late;         // whether a late value is no number (SmemState::late)
};

// One request's work tiles.
struct Request {
  int row0, n, ctx;   // first row, new tokens, keys before them
  bool dead;          // no keys: one unit per work tile
  int qn;             // work tiles per key/value head
};

// a / b, in 32 bits where both fit (a 64-bit division is a subroutine).
__device__ __forceinline__ long long div_ll(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// Request r; r == R is the padding rows.  Lengths out of range are reported once per call
// (`report`) and leave a request without keys or without rows.
__device__ __forceinline__ Request load_request(const PagedParams& p, int r, bool report) {
  Request q;
  const int a = p.row_start[r], b = r < p.R ? p.row_start[r + 1] : p.T;
  const bool rows_ok = a >= 0 && a <= b && b <= p.T && (r > 0 || a == 0);
  const int kv = r < p.R ? p.kv_len[r] : 0;
  const bool kv_ok = kv <= (p.max_pages << p.page_shift);
  if (report && !(rows_ok && kv_ok)) atomicOr(p.status, kDevCheck);
  q.row0 = a;
  q.n = rows_ok ? b - a : 0;
  q.dead = !kv_ok || kv < q.n || r == p.R;
  q.ctx = q.dead ? 0 : kv - q.n;
  q.qn = (q.n + (1 << p.tQ_shift) - 1) >> p.tQ_shift;
  return q;
}

// Key tiles of the request's first k work tiles, all full (tQ = 2 tq tokens: pairs), and two
// units for each: tile i reaches position ctx + (i + 1) tQ.  With tQ dividing 128,
// ceil((ctx + (i + 1) tQ) / 128) = ceil((c0 + i + 1) / P) for c0 = ceil(ctx / tQ) and
// P = 128 / tQ, and the sum over i is a difference of sums of ceil(m / P); with tQ = 256 a
// tile adds two key tiles to the last.
__device__ __forceinline__ long long units_of_full(const Request& q, long long k, int tQ_shift) {
  if (q.dead) return 3 * k;
  if (tQ_shift > 7) return k * (k + 1) + k * ((q.ctx + BK - 1) >> 7) + 2 * k;
  const int ps = 7 - tQ_shift;
  const long long c0 = (q.ctx + (1 << tQ_shift) - 1) >> tQ_shift;
  auto sum = [ps](long long n) {
    const long long d = n >> ps, rem = n & ((1 << ps) - 1);
    return ((d * (d + 1)) >> 1 << ps) + rem * (d + 1);
  };
  return sum(c0 + k) - sum(c0) + 2 * k;
}
__device__ __forceinline__ int key_tiles(const Request& q, int i, int tQ_shift) {
  return q.dead ? 1 : (q.ctx + min(q.n, (i + 1) << tQ_shift) + BK - 1) >> 7;
}
// Units that work tile i counts beyond its key tiles: two with tokens in both halves.
__device__ __forceinline__ int extra_units(const Request& q, int i, int tQ_shift) {
  return q.n - (i << tQ_shift) > 1 << (tQ_shift - 1) ? 2 : 1;
}
// Units of one key/value head of the request.
__device__ __forceinline__ long long head_units(const Request& q, int tQ_shift) {
  if (q.qn == 0) return 0;
  const int last = q.qn - 1, units = key_tiles(q, last, tQ_shift) + extra_units(q, last, tQ_shift);
  return last == 0 ? units : units_of_full(q, last, tQ_shift) + units;
}

// Descriptor of a key or value tile in shared memory: [16 groups][2 halves][8 rows][64] bf16,
// 128-byte swizzle, as one box per page lays it down whatever the page's size.  A group of eight
// keys and the next are 2048 bytes apart (the stride byte offset: along N for the keys, which are
// K-major, along K for the values, which are MN-major), a half and the other 1024 (the leading
// byte offset of the values' 64-column atoms).
__device__ __forceinline__ uint64_t kv_desc(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | static_cast<uint64_t>(1024 >> 4) << 16 |
         static_cast<uint64_t>(2048 >> 4) << 32 | static_cast<uint64_t>(1) << 46 | static_cast<uint64_t>(2) << 61;
}

struct SmemState {
  uint64_t q_full[2], q_empty[2];
  uint64_t ring_full[STAGES], ring_empty[STAGES];
  uint64_t s_full[4];    // pair: half 0, 1; single: even, odd key tile
  uint64_t p_full[2];    // single: even, odd key tile
  uint64_t pv_done[2];   // single: even, odd key tile
  uint64_t o_full[2];
  uint64_t item_full[ITEMS], item_empty[ITEMS];
  Item items[ITEMS];
  // Of an item and column, the first of the values that only some rows of the work tile see and
  // that are NaN (byte 0), +inf (1), -inf (2): 256 less its position after the tile's first token;
  // 0: none.
  alignas(16) uint32_t late[ITEMS][HD];
  long long warp_sum[WARPS];
  long long start_off;   // units of the starting request before the range
  int start_req;
  int dead;              // the issuer has given up
  Request start;
  uint32_t tmem;
};
static_assert(sizeof(SmemState) <= SMEM_BYTES - STATE_OFF, "the state fits behind the ring");

// A ring stage and the parity of its use; the next one.
struct Ring {
  uint32_t stage, phase;
  __device__ __forceinline__ Ring next() const {
    return stage + 1 == STAGES ? Ring{0, phase ^ 1u} : Ring{stage + 1, phase};
  }
};

__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(e));
  return e != 0;
}

// Whether three phases are done (give one twice for two); the tests are on their way together.
__device__ __forceinline__ bool mbar_test_all(uint32_t b0, uint32_t p0, uint32_t b1, uint32_t p1, uint32_t b2,
                                              uint32_t p2) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q, r;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 q, [%3], %4;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 r, [%5], %6;\n\t"
      "and.pred p, p, q;\n\t"
      "and.pred p, p, r;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(b0), "r"(p0), "r"(b1), "r"(p1), "r"(b2), "r"(p2)
      : "memory");
  return ok != 0;
}
// Bounded wait of a warp for three phases; every lane tests, and all have the same outcome.
__device__ __forceinline__ bool warp_wait_all(uint32_t b0, uint32_t p0, uint32_t b1, uint32_t p1, uint32_t b2,
                                              uint32_t p2, int* status) {
  unsigned long long t0 = 0;
  while (true) {
    for (int i = 0; i < 256; ++i)
      if (__all_sync(FULL, mbar_test_all(b0, p0, b1, p1, b2, p2))) return true;
    const unsigned long long now = globaltimer_ns();
    if (t0 == 0) t0 = now;
    if (__any_sync(FULL, now - t0 > kWaitLimitNs)) {
      atomicOr(status, kDevTimeout);
      return false;
    }
  }
}

// Warp-wide wait by lane 0.
__device__ __forceinline__ bool warp_wait(const uint64_t* bar, uint32_t parity, int* status) {
  int w = 1;
  if (threadIdx.x % 32 == 0) w = mbar_wait(smem_u32(bar), parity & 1u, status) ? 1 : 0;
  w = __shfl_sync(FULL, w, 0);
  __syncwarp();  // what lane 0 acquired is every lane's
  return w != 0;
}

// The same for the eight warps of a query half (hardware barrier 1 + wg): one lane of the first
// warp polls, the others sleep at the barrier, which hands them the outcome; sixteen polling warps
// slow the loading and the issuing warp down (a call's start: 2.4 us to the first score product
// instead of 1.7).  With `dead` the wait gives up, past its limit, only once the issuer has: the
// issuer's waits for the parts of P have no limit of their own, and end because a half that has an
// item hands over every part of it.
// TRIES tests in a row before the clock is read; for the scores 32 measured best (a test per loop
// 137 us, 4 or 8 133, 32 or 64 127 for the 2 x 2011 tokens), where the wait is once per item the
// short code does (its instructions are fetched anew by every launch).
template <int TRIES>
__device__ __forceinline__ uint32_t poll(uint32_t bar, uint32_t parity, int* status, const int* dead) {
  if (mbar_try_wait(bar, parity)) return 1;
  const unsigned long long t0 = globaltimer_ns();
  while (true) {
#pragma unroll
    for (int i = 0; i < TRIES; ++i)
      if (mbar_try_wait(bar, parity)) return 1;
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      atomicOr(status, kDevTimeout);
      if (!dead || *(const volatile int*)dead) return 0;
    }
  }
}
template <int TRIES = 4>
__device__ __forceinline__ bool half_wait(const uint64_t* bar, uint32_t parity, int wg, int* status, const int* dead) {
  uint32_t ok = 1;
  if (threadIdx.x % 256 == 0) ok = poll<TRIES>(smem_u32(bar), parity & 1u, status, dead);
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred q, %2, 256, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(ok)
      : "r"(ok), "r"(1 + wg)
      : "memory");
  return ok != 0;
}

// Hardware barriers between the eight warps of a query half, which arrive, and the issuing warp,
// which waits: no test of a barrier in shared memory, which takes some 250 cycles while the tensor
// pipe reads operands there.  In the form that counts threads: no warp has to be converged.
__device__ __forceinline__ void part_arrive(int id) {
  __syncwarp();
  asm volatile("barrier.cta.arrive %0, 288;" ::"r"(id) : "memory");
}
__device__ __forceinline__ void part_wait(int id) {
  __syncwarp();
  asm volatile("barrier.cta.sync %0, 288;" ::"r"(id) : "memory");
}

// TMEM in the 16 x 256-bit shape: sixteen rows, `n` groups of eight fp32 columns; a lane holds
// columns 2 (lane % 4) + {0, 1} of every group of rows lane / 4 (registers 4 g, 4 g + 1) and
// lane / 4 + 8 (4 g + 2, 4 g + 3).
__device__ __forceinline__ void tmem_ld_quad4(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// Wait for this warp's TMEM loads; the registers they fill are operands, so that nothing that
// uses them moves before it.
__device__ __forceinline__ void tmem_wait_quad4(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_wait_quad4(uint32_t (&r)[16], uint32_t (&q)[16]) {
  tmem_wait_quad4(r);
  asm volatile(""
               : "+r"(q[0]), "+r"(q[1]), "+r"(q[2]), "+r"(q[3]), "+r"(q[4]), "+r"(q[5]), "+r"(q[6]), "+r"(q[7]),
                 "+r"(q[8]), "+r"(q[9]), "+r"(q[10]), "+r"(q[11]), "+r"(q[12]), "+r"(q[13]), "+r"(q[14]), "+r"(q[15])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_st_quad4(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// The 16 x 128-bit shape, four groups of four 32-bit columns: column lane % 4 of every group of
// rows lane / 4 (register 2 g) and lane / 4 + 8 (2 g + 1): the bf16 pairs of the shape above.
__device__ __forceinline__ void tmem_st_pairs4(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}

// Whether one of two bf16 (of eight) has the exponent of NaN and infinity, in bits 15 and 31.
__device__ __forceinline__ uint32_t no_number(uint32_t w) { return (w & 0x7F807F80u) + 0x00800080u; }
__device__ __forceinline__ bool no_number(const uint4& v) {
  return ((no_number(v.x) | no_number(v.y) | no_number(v.z) | no_number(v.w)) & 0x80008000u) != 0;
}
// Takes what is no number out of half a value row in shared memory (64 columns from `col0` on, 16-byte
// chunks xor `swizzle`) and notes it under `mark`, 256 less the row's position after the work tile's
// first token.  The note is there before the value is gone: a thread of the other query half that
// finds the row clean finds the note.
__device__ __noinline__ void take_out(uint4* row, int swizzle, int col0, uint32_t mark, uint32_t* late, int* any) {
  *any = 1;
  for (int c = 0; c < 8; ++c) {
    uint4 v = row[c];
    if (!no_number(v)) continue;
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
    for (int e = 0; e < 8; ++e) {
      const uint32_t h = w[e >> 1] >> (16 * (e & 1)) & 0xFFFFu;
      if ((h & 0x7F80u) != 0x7F80u) continue;
      const uint32_t note = mark << (h & 0x7Fu ? 0 : h >> 15 ? 16 : 8);
      uint32_t* const at = late + col0 + ((c ^ swizzle) << 3) + e;
      // The larger of each byte; a turn that fails means that another thread raised one.
      for (uint32_t was = *(volatile uint32_t*)at, old; (old = atomicCAS(at, was, __vmaxu4(was, note))) != was; was = old) {
      }
      w[e >> 1] &= e & 1 ? 0x0000FFFFu : 0xFFFF0000u;
    }
    __threadfence_block();
    row[c] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
// Adds the values taken out to the warp's rows (`tok`: their tokens in the work tile) that see them.
__device__ __noinline__ void add_late(const uint32_t* late, uint32_t ocol, int tok0, int tok1) {
  for (int y = 0; y < HD / 32; ++y) {
    uint32_t o[16];
    tmem_ld_quad4(ocol + 32 * y, o);
    tmem_wait_quad4(o);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t n = late[32 * y + (i >> 2) * 8 + (threadIdx.x & 3) * 2 + (i & 1)];
      const uint32_t tok = i & 2 ? tok1 : tok0;
      const bool nan = (n & 0xFFu) + tok >= 256, up = (n >> 8 & 0xFFu) + tok >= 256, down = (n >> 16) + tok >= 256;
      if (nan || up || down) {
        const float v = nan || (up && down) ? NAN : up ? INFINITY : -INFINITY;
        o[i] = __float_as_uint(__uint_as_float(o[i]) + v);
      }
    }
    __syncwarp();
    tmem_st_quad4(ocol + 32 * y, o);
  }
  tmem_wait_st();
}

__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(FULL, x, 1));
  return fmaxf(x, __shfl_xor_sync(FULL, x, 2));
}
__device__ __forceinline__ float quad_sum(float x) {
  x += __shfl_xor_sync(FULL, x, 1);
  return x + __shfl_xor_sync(FULL, x, 2);
}

// Adds another CTA's part of the warp's sixteen rows to the warp's own: O in TMEM, m and l.
// The same rows are the same warp's in every CTA, so a warp waits for a warp.  Bounded; on a
// timeout the status word is set and the warp goes on (its output is then unspecified).
__device__ __forceinline__ void add_part(const uint8_t* part, unsigned long long* flag, unsigned long long call,
                                         int* status, int prow, uint32_t valid, uint32_t ocol, float (&m)[2],
                                         float (&l)[2]) {
  const int lane = threadIdx.x % 32;
  if (lane == 0) {
    unsigned long long t0 = 0, v;
    while (true) {
      asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(flag) : "memory");
      if (v == call) break;
      const unsigned long long now = globaltimer_ns();
      if (t0 == 0) {
        t0 = now;
      } else if (now - t0 > kWaitLimitNs) {
        atomicOr(status, kDevTimeout);
        break;
      }
      __nanosleep(64);
    }
    *flag = 0;
  }
  __syncwarp();
  __threadfence();
  const float* const ml = reinterpret_cast<const float*>(part + PART_O) + prow;
  const float2* const po = reinterpret_cast<const float2*>(part) + prow * 4 + (lane & 3);
  float f[2], w[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const bool in = valid >> x & 1;
    const float mo = in ? __ldcg(ml + 8 * x) : -INFINITY, lo = in ? __ldcg(ml + 256 + 8 * x) : 0.f;
    const float top = fmaxf(m[x], mo);
    f[x] = m[x] == top ? 1.f : ex2(m[x] - top);
    w[x] = mo == -INFINITY ? 0.f : ex2(mo - top);
    m[x] = top;
    l[x] = f[x] * l[x] + w[x] * lo;
  }
#pragma unroll 1
  for (int y = 0; y < HD / 32; ++y) {
    uint32_t o[16];
    tmem_ld_quad4(ocol + 32 * y, o);
    float2 v[8];  // a weight of 0 (a row without keys in that part) hides what it holds
#pragma unroll
    for (int k = 0; k < 8; ++k)
      v[k] = w[k & 1] != 0.f ? __ldcg(po + (y * 4 + (k >> 1)) * 1024 + (k & 1) * 32) : make_float2(0.f, 0.f);
    __syncwarp();
    tmem_wait_quad4(o);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float g = f[k & 1], h = w[k & 1];
      o[2 * k] = __float_as_uint(fmaf(h, v[k].x, g != 0.f ? g * __uint_as_float(o[2 * k]) : 0.f));
      o[2 * k + 1] = __float_as_uint(fmaf(h, v[k].y, g != 0.f ? g * __uint_as_float(o[2 * k + 1]) : 0.f));
    }
    tmem_st_quad4(ocol + 32 * y, o);
  }
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__global__ void __launch_bounds__(THREADS, 1) paged_attention_kernel(const __grid_constant__ PagedParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  SmemState& sm = *reinterpret_cast<SmemState*>(smem + STATE_OFF);
  const uint32_t base = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  if (base & 1023u) {  // the swizzled tiles need it; the declaration asks for it
    if (tid == 0) {
      atomicOr(p.status, kDevCheck);
      pdl_wait();
      p.splits[blockIdx.x] = Split{0, 0, 0, -1};  // nothing for paged_combine_kernel to join
    }
    return;
  }

  if (warp == LOAD_WARP && lane == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sm.q_full[i]), 1);
      mbar_init(smem_u32(&sm.q_empty[i]), 1);
      mbar_init(smem_u32(&sm.pv_done[i]), 1);
      mbar_init(smem_u32(&sm.o_full[i]), 1);
    }
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(smem_u32(&sm.ring_full[i]), 1);
      mbar_init(smem_u32(&sm.ring_empty[i]), 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_u32(&sm.s_full[i]), 1);
      if (i < 2) mbar_init(smem_u32(&sm.p_full[i]), SOFTMAX_WARPS / 2);
    }
    for (int i = 0; i < ITEMS; ++i) {
      mbar_init(smem_u32(&sm.item_full[i]), 1);
      mbar_init(smem_u32(&sm.item_empty[i]), 1 + SOFTMAX_WARPS);  // the issuer and the softmax warps
    }
    sm.dead = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.q);
    tma_prefetch_desc(&p.k);
    tma_prefetch_desc(&p.v);
  }
  if (warp == MMA_WARP) {
    tmem_alloc(smem_u32(&sm.tmem), TMEM_COLS);
    tmem_relinquish();
  }
  pdl_wait();  // lengths, tables, queries and pages come from earlier kernels
  pdl_trigger();

  // ---------------------------------------------------------------- this CTA's range
  const int nreq = p.R + 1;  // the padding rows last
  const int per = (nreq + THREADS - 1) / THREADS;
  const int r0 = min(nreq, tid * per), r1 = min(nreq, r0 + per);
  long long mine = 0;
  Request req{};  // the thread's last request: with up to 575 of them its only one
  for (int r = r0; r < r1; ++r) {
    req = load_request(p, r, blockIdx.x == 0);
    mine += head_units(req, p.tQ_shift) * p.n_kv_head;
  }
  long long upto = mine;
#pragma unroll 1  // short code: its instructions are fetched for one use
  for (int o = 1; o < 32; o <<= 1) {
    const long long up = __shfl_up_sync(FULL, upto, o);
    if (lane >= o) upto += up;
  }
  if (lane == 31) sm.warp_sum[warp] = upto;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  long long total = 0;
#pragma unroll 1
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) upto += sm.warp_sum[w];
    total += sm.warp_sum[w];
  }
  const int ctas = (int)min((long long)gridDim.x, total);  // every range holds a unit
  const int c = blockIdx.x;
  const bool working = c < ctas;
  const bool one = total == ctas;  // a unit each: no division
  const long long u0 = !working ? 0 : one ? c : div_ll(total * c, ctas);
  const long long u1 = !working ? 0 : one ? c + 1 : div_ll(total * (c + 1), ctas);
  if (working && mine > 0 && u0 >= upto - mine && u0 < upto) {
    long long at = upto - mine;
    int r = r0;
    if (per > 1) {
      while (true) {
        req = load_request(p, r, false);
        const long long units = head_units(req, p.tQ_shift) * p.n_kv_head;
        if (u0 < at + units) break;
        at += units;
        ++r;
      }
    }
    sm.start = req;
    sm.start_req = r;
    sm.start_off = u0 - at;
  }
  __syncthreads();
  const uint32_t tmem = sm.tmem;

  if (warp == LOAD_WARP) {
    // ------------------------------------------------------------ walk and TMA copies
    const int nb = BK >> p.page_shift;         // pages per key tile
    const int box = lane & (nb - 1);
    const bool copies = lane < nb;
    const uint32_t box_dst = (box << p.page_shift) * 256;
    const uint32_t q_bytes = (uint32_t)(2 * p.tq * p.G * 128);
    const int rows_end = (int)(((long long)p.pages * p.n_kv_head << p.page_shift) >> 3);  // out of range: zeros
    int r = working ? sm.start_req : 0;
    long long off = working ? sm.start_off : 0;
    Request q = sm.start;
    int g = 0;
    int i = 0;  // the work tile that holds unit `off` of the head: units_of_full(i) <= off
    if (working) {
      if (p.n_kv_head > 1) {
        const long long units = head_units(q, p.tQ_shift);
        while (off >= units) {
          off -= units;
          ++g;
        }
      }
      int hi = q.qn;
      while (hi - i > 1) {
        const int mid = (i + hi) >> 1;
        if (units_of_full(q, mid, p.tQ_shift) <= off) i = mid;
        else hi = mid;
      }
    }
    int j = (int)(off - units_of_full(q, i, p.tQ_shift));
    long long unit = u0;
    uint32_t items = 0, loads = 0, q_uses[2] = {0, 0};
    int next_half = 0;
    Split split{0, 0, 0, -1};
    bool ok = true;
    while (ok && unit < u1) {
      const int tile_n = key_tiles(q, i, p.tQ_shift);
      const int units = (int)min((long long)(tile_n + extra_units(q, i, p.tQ_shift) - j), u1 - unit);  // in the range
      Item it;
      it.row0 = q.row0 + (i << p.tQ_shift);
      it.ntok = min(1 << p.tQ_shift, q.n - (i << p.tQ_shift));
      it.pos0 = q.ctx + (i << p.tQ_shift);
      it.kvlim = q.dead ? 0 : it.pos0 + it.ntok;
      it.j0 = j;
      it.nt = min(units, tile_n - j);  // the units past the key tiles hold no work
      it.g = g;
      it.late = 0;
      if (it.nt > 0) {
        // Page ids of the first key tile.
        const int32_t* const row = p.table + (long long)r * p.max_pages;
        auto page_id = [&](int t) {  // -1: no key there that the tile may see
          const int page = (it.j0 + t) * nb + box;
          return copies && ((long long)page << p.page_shift) < it.kvlim ? row[page] : -1;
        };
        int id = page_id(0);
        it.half = it.ntok > p.tq ? 2 : next_half;
        const bool ends = j + it.nt == tile_n;
        it.part = -1;
        it.added = 0;
        if (j > 0 || !ends) {  // unit u belongs to CTA ((u + 1) ctas - 1) / total
          const int cf = j == 0 ? c : (int)div_ll((unit - j + 1) * ctas - 1, total);
          const int cl = ends ? c : (int)div_ll((unit - j + tile_n) * ctas - 1, total);
          if (cl - cf <= (it.half == 2 ? MOST_ADDED : 0)) it.added = cl - cf;
          if (j > 0 || it.added == 0) it.part = j == 0 ? 2 * c + 1 : 2 * c;
          if (j == 0 && it.added == 0) split = Split{it.row0, it.ntok, g, cl};
        }
        // The query halves, while the page ids are on their way.
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!ok || (it.half != 2 && it.half != h)) continue;
          ok = warp_wait(&sm.q_empty[h], q_uses[h] ^ 1u, p.status);
          if (!ok) continue;
          if (lane == 0) {
            const uint32_t qbar = smem_u32(&sm.q_full[h]);
            mbar_arrive_expect_tx(qbar, q_bytes);
            const int tok = it.row0 + (it.half == 2 ? h * p.tq : 0);
            tma_load_4d(base + h * TILE_BYTES, &p.q, qbar, 0, 0, g * p.G, tok);
            tma_load_4d(base + h * TILE_BYTES + ATOM_BYTES, &p.q, qbar, 0, 1, g * p.G, tok);
          }
          ++q_uses[h];
        }
        // The key and value tiles, one box per page and lane.
        for (int t = 0; t < it.nt && ok; ++t) {
          const bool there = ((long long)((it.j0 + t) * nb + box) << p.page_shift) < it.kvlim;
          int coord = rows_end;
          if (copies && there) {
            if (id >= 0 && id < p.pages) coord = (id * p.n_kv_head + g) << (p.page_shift - 3);
            else atomicOr(p.status, kDevCheck);
          }
          if (t + 1 < it.nt) id = page_id(t + 1);
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const int st = loads % STAGES;
            if (!warp_wait(&sm.ring_empty[st], (loads / STAGES) ^ 1u, p.status)) {
              ok = false;
              break;
            }
            const uint32_t bar = smem_u32(&sm.ring_full[st]);
            if (lane == 0) mbar_arrive_expect_tx(bar, TILE_BYTES);
            __syncwarp();
            if (copies)
              tma_load_4d(base + RING_OFF + st * TILE_BYTES + box_dst, kv ? &p.v : &p.k, bar, 0, 0, 0, coord);
            ++loads;
            if (t == 0 && kv == 0) {  // the item, behind its first key tile
              const int slot = items % ITEMS;
              ok = warp_wait(&sm.item_empty[slot], (items / ITEMS) ^ 1u, p.status);
              if (!ok) break;
              reinterpret_cast<uint4*>(sm.late[slot])[lane] = make_uint4(0, 0, 0, 0);
              __syncwarp();
              if (lane == 0) {
                sm.items[slot] = it;
                mbar_arrive(smem_u32(&sm.item_full[slot]));
              }
              __syncwarp();
              ++items;
            }
          }
        }
        if (it.half != 2) next_half = it.half ^ 1;
      }
      unit += units;
      // The next work tile: query tile, then head, then request.
      if (unit < u1) {
        j = 0;
        if (++i == q.qn) {
          i = 0;
          if (++g == p.n_kv_head) {
            g = 0;
            do q = load_request(p, ++r, false);
            while (q.qn == 0);
          }
        }
      }
    }
    if (lane == 0) p.splits[c] = split;
    if (ok) {  // nt == 0 ends the walk
      const int slot = items % ITEMS;
      if (warp_wait(&sm.item_empty[slot], (items / ITEMS) ^ 1u, p.status) && lane == 0) {
        sm.items[slot].nt = 0;
        mbar_arrive(smem_u32(&sm.item_full[slot]));
      }
      __syncwarp();
    }
    // No copy may still be landing when the CTA exits.
    for (int h = 0; h < 2; ++h)
      if (q_uses[h]) warp_wait(&sm.q_full[h], q_uses[h] - 1, p.status);
    for (uint32_t l = loads > STAGES ? loads - STAGES : 0; l < loads; ++l)
      warp_wait(&sm.ring_full[l % STAGES], l / STAGES, p.status);
  } else if (warp == MMA_WARP) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp walks the items, so that descriptors are built in uniform registers; one
    // elected lane issues.  A barrier test costs some 250 cycles while the tensor pipe reads
    // shared memory, and the pipe holds about four products (both measured): one test for all
    // that a step needs.
    constexpr uint32_t id_s = idesc_bf16_f32(128, BK, 0, 0);
    constexpr uint32_t id_pv = idesc_bf16_f32(128, HD, 0, 1);
    const bool issues = elect_one();
    uint32_t q_uses[2] = {0, 0}, even = 0, odd = 0;
    Ring key{0, 0};  // of the next key tile; its value tile is the stage behind
    auto score = [&](int half, int buf, uint32_t st) {  // S[buf] = Q[half] K^T
      const uint64_t qd = sw128_kmajor_desc(base + half * TILE_BYTES);
      const uint64_t kd = kv_desc(base + RING_OFF + st * TILE_BYTES);
      if (issues) {
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk)
          tc_mma_bf16(tmem + buf * BK, qd + (kk >> 2) * (ATOM_BYTES >> 4) + 2 * (kk & 3),
                      kd + (kk >> 2) * (1024 >> 4) + 2 * (kk & 3), id_s, kk != 0);
      }
    };
    // O[out] (+)= P[buf] V for `n` steps of 16 keys from step k0 on; `first` of the item's.
    auto value = [&](int out, int buf, uint32_t st, int k0, int n, bool first) {
      const uint64_t vd = kv_desc(base + RING_OFF + st * TILE_BYTES);
      if (issues) {
#pragma unroll
        for (int kk = k0; kk < k0 + n; ++kk)
          tc_mma_bf16_a_tmem(tmem + O_COL + out * HD, tmem + buf * BK + (kk >> 2) * 64 + (kk & 3) * 8,
                             vd + kk * 256u, id_pv, !first || kk != k0);
      }
    };
    auto commit = [&](const uint64_t* bar) {
      if (issues) tc_commit(smem_u32(bar));
    };
    for (uint32_t items = 0;; ++items) {
      const int slot = items % ITEMS;
      if (!warp_wait(&sm.item_full[slot], items / ITEMS, p.status)) {
        sm.dead = 1;
        break;
      }
      const int nt = __shfl_sync(FULL, sm.items[slot].nt, 0), half = __shfl_sync(FULL, sm.items[slot].half, 0);
      if (issues) mbar_arrive(smem_u32(&sm.item_empty[slot]));
      if (nt == 0) break;
      const bool pair = half == 2;
      const uint32_t q0 = smem_u32(&sm.q_full[half == 1]), q0_phase = (half == 1 ? q_uses[1] : q_uses[0]) & 1u;
      const uint32_t q1 = pair ? smem_u32(&sm.q_full[1]) : q0, q1_phase = pair ? q_uses[1] & 1u : q0_phase;
      q_uses[0] += pair || half == 0;
      q_uses[1] += pair || half == 1;
      auto full = [&](const Ring& r) { return smem_u32(&sm.ring_full[r.stage]); };
      if (!warp_wait_all(full(key), key.phase, q0, q0_phase, q1, q1_phase, p.status)) {
        sm.dead = 1;
        break;
      }
      tc_fence_after();
      bool ok = true;
      if (pair) {
        for (int h = 0; h < 2; ++h) {
          score(h, h, key.stage);
          commit(&sm.s_full[h]);
        }
        commit(&sm.ring_empty[key.stage]);
        for (int t = 0; t < nt; ++t) {
          const bool more = t + 1 < nt;
          const Ring val = key.next(), next = val.next(), last = more ? next : val;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            // In front of the first half the value tile and the next key tile; then P in three parts.
            if (h == 0 && !(ok = warp_wait_all(full(val), val.phase, full(last), last.phase, full(last), last.phase,
                                               p.status)))
              break;
            part_wait(PART_BAR + h);
            tc_fence_after();
            value(h, h, val.stage, 4, 4, t == 0);
            part_wait(PART_BAR + 2 + h);
            tc_fence_after();
            value(h, h, val.stage, 0, 2, false);
            part_wait(PART_BAR + 4 + h);
            tc_fence_after();
            value(h, h, val.stage, 2, 2, false);
            if (more) {
              score(h, h, next.stage);
              commit(&sm.s_full[h]);  // covers the value product before it
            } else {
              commit(&sm.o_full[h]);
              commit(&sm.q_empty[h]);
            }
          }
          if (!ok) break;
          commit(&sm.ring_empty[val.stage]);
          if (more) commit(&sm.ring_empty[next.stage]);
          key = next;
        }
      } else {
        score(half, 0, key.stage);
        commit(&sm.s_full[2]);
        commit(&sm.ring_empty[key.stage]);
        if (nt == 1) commit(&sm.q_empty[half]);
        for (int t = 0; t < nt; ++t) {
          // The score product of the next tile and this tile's value product, whichever can go
          // first: a late key tile does not keep the value tile's stage.
          const int b = t & 1;
          const Ring val = key.next(), next = val.next();
          const uint32_t pf = smem_u32(&sm.p_full[b]), pp = ((b ? odd : even) + (t >> 1)) & 1u;
          bool scored = t + 1 == nt, valued = false;
          unsigned long long t0 = 0;
          for (uint32_t polls = 1; !(scored && valued); ++polls) {
            if (!scored && __all_sync(FULL, mbar_test_all(full(next), next.phase, full(next), next.phase, full(next),
                                                          next.phase))) {
              tc_fence_after();
              score(half, b ^ 1, next.stage);
              commit(&sm.s_full[2 + (b ^ 1)]);
              commit(&sm.ring_empty[next.stage]);
              if (t + 2 == nt) commit(&sm.q_empty[half]);  // every score product is issued
              scored = true;
            }
            if (!valued && __all_sync(FULL, mbar_test_all(pf, pp, full(val), val.phase, pf, pp))) {
              tc_fence_after();
              value(0, b, val.stage, 4, 4, t == 0);
              value(0, b, val.stage, 0, 4, false);
              if (t + 1 == nt) commit(&sm.o_full[0]);
              commit(&sm.pv_done[b]);
              commit(&sm.ring_empty[val.stage]);
              valued = true;
            }
            if (polls % 256 == 0) {  // bounded as every wait
              const unsigned long long now = globaltimer_ns();
              if (t0 == 0) t0 = now;
              if (__any_sync(FULL, now - t0 > kWaitLimitNs)) {
                if (issues) atomicOr(p.status, kDevTimeout);
                ok = false;
                break;
              }
            }
          }
          if (!ok) break;
          key = next;
        }
        even += (nt + 1) >> 1;
        odd += nt >> 1;
      }
      if (!ok) {
        sm.dead = 1;
        break;
      }
    }
  } else {
    // ------------------------------------------------------------ softmax warps
    const int wg = warp >> 3;
    const int lane0 = (warp & 3) * 32 + ((warp >> 2) & 1) * 16;  // the warp's sixteen rows of the half
    const int quad = lane & 3;
    const uint32_t tl = tmem + ((uint32_t)lane0 << 16);
    const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
    uint32_t tiles = 0, pairs = 0, even = 0, odd = 0, outs = 0;  // even, odd: a single item's key tiles
    bool ok = true;
    for (uint32_t items = 0; ok; ++items) {
      const int slot = items % ITEMS;
      if (!half_wait(&sm.item_full[slot], items / ITEMS, wg, p.status, &sm.dead)) break;
      const Item& it = sm.items[slot];  // this warp's until it arrives at item_empty
      const int nt = it.nt;
      const bool pair = it.half == 2;
      if (nt == 0 || (!pair && wg == 1)) {
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.item_empty[slot]));
        if (nt == 0) break;
        tiles += nt;
        continue;
      }
      const int kvlim = it.kvlim, first_key = it.j0 * BK;
      const int all_see = min(it.pos0 + 1, kvlim);  // keys that every row of the work tile sees
      // Keys that this lane's rows (lane0 + lane / 4 and eight further) see; a row that is not
      // stored needs no mask.
      int limit[2];
      uint32_t valid = 0;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int tok_in = (lane0 + lane / 4 + 8 * x) / p.G, tok = (pair ? wg * p.tq : 0) + tok_in;
        const bool v = tok_in < p.tq && tok < it.ntok;
        limit[x] = !v ? 0x7FFFFFFF : kvlim ? it.pos0 + tok + 1 : 0;
        valid |= v ? 1u << x : 0u;
      }
      const bool active = __any_sync(FULL, valid != 0);
      const uint32_t ocol = tl + O_COL + (pair ? wg * HD : 0);
      float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
      for (int t = 0; t < nt; ++t) {
        const int b = t & 1;
        const int sb = pair ? wg : 2 + b;            // barrier set
        const uint32_t scol = tl + (pair ? wg : b) * BK;
        const uint32_t ph = pair ? pairs + t : (b ? odd : even) + (t >> 1);
        const int k0 = first_key + t * BK;
        if (k0 + BK > all_see) {
          // Values that some row of the tile does not see: rows all_see - k0 .. 127 of the stage, no
          // row from kvlim - k0 on.  While the tile's scores are computed.
          const uint32_t vl = 2 * (tiles + t) + 1;
          half_wait(&sm.ring_full[vl % STAGES], vl / STAGES, wg, p.status, nullptr);
          const int zrow = tid & 127, zcol = (tid >> 7) & 1;  // one row's 128 bytes per thread of the eight warps
          if (zrow >= all_see - k0) {  // chunk x + zrow: eight rows of a warp take eight bank groups
            uint4* const z = reinterpret_cast<uint4*>(smem + RING_OFF + (vl % STAGES) * TILE_BYTES + (zrow >> 3) * 2048 +
                                                      zcol * 1024 + (zrow & 7) * 128);
            if (zrow >= kvlim - k0) {
#pragma unroll 1
              for (int x = 0; x < 8; ++x) z[(x + zrow) & 7] = make_uint4(0, 0, 0, 0);
              fence_proxy_async_smem();
            } else {
              bool found = false;
#pragma unroll 4
              for (int x = 0; x < 8; ++x) found |= no_number(z[(x + zrow) & 7]);
              if (__builtin_expect(found, 0)) {
                take_out(z, zrow & 7, 64 * zcol, 256 - (k0 + zrow - it.pos0), sm.late[slot], &sm.items[slot].late);
                fence_proxy_async_smem();
              }
            }
          }
          __syncwarp();
        }
        if (!half_wait<32>(&sm.s_full[sb], ph, wg, p.status, &sm.dead)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (active) {
          // The maximum needs all 128 keys, in two loads of 64; the second one's stay in
          // registers, the first one's are read again for their exponentials, 32 keys at a time
          // behind the arithmetic (96 registers a thread, for 16 warps).
          const bool edge = __any_sync(FULL, min(limit[0], limit[1]) < k0 + BK);
          uint32_t va[16], vb[16];  // 32 keys each
          auto mask = [&](uint32_t(&v)[16], int y) {
            if (edge) {
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if (k0 + 32 * y + (i >> 2) * 8 + quad * 2 + (i & 1) >= limit[(i >> 1) & 1])
                  v[i] = __float_as_uint(-INFINITY);
            }
          };
          auto row_max = [&](const uint32_t(&v)[16], int x) {
            float mx[2];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float a = fmaxf(__uint_as_float(v[4 * i + 2 * x]), __uint_as_float(v[4 * i + 2 * x + 1]));
              mx[i & 1] = i < 2 ? a : fmaxf(mx[i & 1], a);
            }
            return fmaxf(mx[0], mx[1]);
          };
          float tmax[2];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            tmem_ld_quad4(scol + 64 * y, va);
            tmem_ld_quad4(scol + 64 * y + 32, vb);
            tmem_wait_quad4(va, vb);
            mask(va, 2 * y);
            mask(vb, 2 * y + 1);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const float a = fmaxf(row_max(va, x), row_max(vb, x));
              tmax[x] = y ? fmaxf(tmax[x], a) : a;
            }
          }
          // The scale is positive: the maximum commutes with it.
          tmax[0] = quad_max(tmax[0]) * p.scale_log2;
          tmax[1] = quad_max(tmax[1]) * p.scale_log2;
          float factor[2] = {1.0f, 1.0f};
          bool grow = false;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (t == 0) {
              m[x] = tmax[x];
            } else if (tmax[x] > m[x] + 8.0f) {
              factor[x] = ex2(m[x] - tmax[x]);
              m[x] = tmax[x];
              grow = true;
            }
          }
          if (__any_sync(FULL, grow)) {
            // Every earlier value product has to be done: a pair's score commit covers it.  A wait
            // that gives up has set the status; the warp goes on, since its half waits together.
            if (!pair) warp_wait(&sm.pv_done[b ^ 1], (b ? even : odd) + ((t - 1) >> 1), p.status);
            tc_fence_after();
            l[0] *= factor[0];
            l[1] *= factor[1];
#pragma unroll 1
            for (int x = 0; x < HD / 32; ++x) {
              uint32_t o[16];
              tmem_ld_quad4(ocol + 32 * x, o);
              tmem_wait_quad4(o);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * factor[(i >> 1) & 1]);
              tmem_st_quad4(ocol + 32 * x, o);
            }
            tmem_wait_st();
          }
          // 2^(s scale - m); a row without keys so far has m = -inf and only masked scores.
          const float mu0 = m[0] == -INFINITY ? 0.f : -m[0], mu1 = m[1] == -INFINITY ? 0.f : -m[1];
          float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          auto weights = [&](const uint32_t(&v)[16], int y) {  // P of 32 keys, over the scores of half y / 2
            uint32_t pk[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int x = i & 1;
              const float mu = x ? mu1 : mu0;
              const float2 a = __ffma2_rn(make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), sc2,
                                          make_float2(mu, mu));
              const float2 e = make_float2(ex2(a.x), ex2(a.y));
              ls[x] = __fadd2_rn(ls[x], e);
              pk[i] = pack_bf16x2(e.x, e.y);
            }
            tmem_st_pairs4(scol + (y >> 1) * 64 + (y & 1) * 16, pk);
          };
          // P of keys 64 .. 127 lies over their own scores (columns 64 .. 95); P of keys 0 .. 63
          // over columns 0 .. 31, whose scores are in registers by then.
          weights(va, 2);
          tmem_ld_quad4(scol, va);
          weights(vb, 3);
          if (pair) {
            tmem_wait_st();
            tc_fence_before();
            part_arrive(PART_BAR + wg);
          }
          tmem_ld_quad4(scol + 32, vb);
          tmem_wait_quad4(va, vb);
          mask(va, 0);
          mask(vb, 1);
          weights(va, 0);
          if (pair) {
            tmem_wait_st();
            tc_fence_before();
            part_arrive(PART_BAR + 2 + wg);
          }
          weights(vb, 1);
          l[0] += ls[0].x + ls[0].y;
          l[1] += ls[1].x + ls[1].y;
          tmem_wait_st();  // P is in TMEM before the MMA may read it
        }
        tc_fence_before();
        if (pair) {
          if (!active) {
            part_arrive(PART_BAR + wg);
            part_arrive(PART_BAR + 2 + wg);
          }
          part_arrive(PART_BAR + 4 + wg);
        } else {
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sm.p_full[b]));
        }
      }
      if (!ok) break;
      tiles += nt;
      if (pair) {
        pairs += nt;
      } else {
        even += (nt + 1) >> 1;
        odd += nt >> 1;
      }
      // ---- the item's output: O / l, or the partial
      l[0] = quad_sum(l[0]);
      l[1] = quad_sum(l[1]);
      auto put_late = [&] {
        const int first = pair ? wg * p.tq : 0, row = lane0 + lane / 4;
        if (__builtin_expect(it.late, 0)) add_late(sm.late[slot], ocol, first + row / p.G, first + (row + 8) / p.G);
      };
      const bool adds = it.added && it.part < 0;
      if (__builtin_expect(adds, 0)) {
        if (!half_wait(&sm.o_full[wg], outs, wg, p.status, &sm.dead)) break;
        tc_fence_after();
        if (active) {
          put_late();
          for (int i = 1; i <= it.added; ++i)
            add_part(p.parts + (size_t)(2 * (blockIdx.x + i)) * PART_BYTES,
                     p.flags + (blockIdx.x + i) * SOFTMAX_WARPS + warp, p.call, p.status,
                     (pair ? wg * 128 : 0) + lane0 + lane / 4, valid, ocol, m, l);
        }
      }
      float inv[2];
      uint16_t* dst[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        inv[x] = l[x] != 0.f ? 1.0f / l[x] : 0.f;  // 0: no keys; a NaN among the scores stays one
        const int mr = lane0 + lane / 4 + 8 * x, tok_in = mr / p.G;
        const long long row = (long long)(it.row0 + (pair ? wg * p.tq : 0) + tok_in) * p.n_head + it.g * p.G +
                              (mr - tok_in * p.G);
        dst[x] = p.out + row * HD + quad * 8;
        if (it.part < 0 && (valid >> x & 1) && p.lse && quad == 0)
          p.lse[row] = l[x] != 0.f ? (m[x] + log2f(l[x])) * LN2 : -INFINITY;
      }
      if (!adds && !half_wait(&sm.o_full[wg], outs, wg, p.status, &sm.dead)) break;
      ++outs;
      tc_fence_after();
      if (active) {
        if (!adds) put_late();
        if (it.part < 0) {
          auto store = [&](const uint32_t(&o)[16], int y) {  // 32 columns: four groups of eight
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              uint32_t w[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                w[i] = inv[x] != 0.f ? pack_bf16x2(__uint_as_float(o[4 * i + 2 * x]) * inv[x],
                                                  __uint_as_float(o[4 * i + 2 * x + 1]) * inv[x])
                                     : 0u;
              // Four lanes hold one pair each of each of four groups; lane i of the quad is to have
              // group i whole: a 4 x 4 transposition, so that a lane stores 16 bytes and a quad 64
              // of its row.
              uint32_t u[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int gsel = quad ^ k;
                const uint32_t send = gsel & 2 ? (gsel & 1 ? w[3] : w[2]) : (gsel & 1 ? w[1] : w[0]);
                u[k] = __shfl_xor_sync(FULL, send, k);  // from lane quad ^ k its pair of group `quad`
              }
              const uint32_t a0 = quad & 1 ? u[1] : u[0], a1 = quad & 1 ? u[0] : u[1];
              const uint32_t a2 = quad & 1 ? u[3] : u[2], a3 = quad & 1 ? u[2] : u[3];
              const uint4 line = quad & 2 ? make_uint4(a2, a3, a0, a1) : make_uint4(a0, a1, a2, a3);
              if (valid >> x & 1) *reinterpret_cast<uint4*>(dst[x] + y * 32) = line;
            }
            __syncwarp();
          };
          uint32_t oa[16], ob[16];  // the next columns load while these are stored
          tmem_ld_quad4(ocol, oa);
#pragma unroll
          for (int y = 0; y < HD / 32; y += 2) {
            tmem_wait_quad4(oa);
            tmem_ld_quad4(ocol + 32 * (y + 1), ob);
            store(oa, y);
            tmem_wait_quad4(ob);
            if (y + 2 < HD / 32) tmem_ld_quad4(ocol + 32 * (y + 2), oa);
            store(ob, y + 1);
          }
        } else {
          uint8_t* const part = p.parts + (size_t)it.part * PART_BYTES;
          const int prow = (pair ? wg * 128 : 0) + lane0 + lane / 4;
          float2* const po = reinterpret_cast<float2*>(part) + prow * 4 + quad;
#pragma unroll 1
          for (int y = 0; y < HD / 32; ++y) {
            uint32_t o[16];
            tmem_ld_quad4(ocol + 32 * y, o);
            tmem_wait_quad4(o);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (valid >> (i & 1) & 1)
                po[(y * 4 + (i >> 1)) * 1024 + (i & 1) * 32] =
                    make_float2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1]));
            __syncwarp();
          }
          float* const ml = reinterpret_cast<float*>(part + PART_O) + prow;
#pragma unroll
          for (int x = 0; x < 2; ++x)
            if ((valid >> x & 1) && quad == 0) {
              ml[8 * x] = m[x];
              ml[256 + 8 * x] = l[x];
            }
          if (it.added) {
            __threadfence();
            __syncwarp();
            if (lane == 0) atomicExch(p.flags + blockIdx.x * SOFTMAX_WARPS + warp, p.call);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.item_empty[slot]));
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

// Joins the partials of the work tile that begins in range blockIdx.y and ends in a later one:
// out = sum_p 2^(m_p - M) O_p / sum_p 2^(m_p - M) l_p over its parts in the order of the keys
// (slot 2 c + 1 of the first CTA, slots 2 c of the others), in one pass with the running M.
// Eight blocks per work tile: of 32 rows each, or, where it has no more rows than that (a decode
// token has G, and up to 152 parts), of two column groups each; there `share` threads share an
// element, every n-th part each, and their sums are joined in a fixed order.  A thread keeps to
// one row, so it needs no one else's weights.  Bound by latency: the launch, the instructions'
// own first fetch, two dependent loads; 2 to 5 us of a call (one token over 131070 keys, whose
// tile has 76 parts: 33.5 us in all), so the code is short: with the parts' weights in shared
// memory first and their sum after, twice the instructions, the 13 x 5 token step took 17.7 us
// instead of 15.0.
constexpr int COMBINE_THREADS = 256;
constexpr int COMBINE_BLOCKS = 8;
struct Joined {  // of some parts: running maximum, sum, weighted O
  float top, sum;
  float4 o;
};
__device__ __forceinline__ void join(Joined& a, float m, float l, const float4& x) {
  const float next = fmaxf(a.top, m);
  if (next == -INFINITY) {  // no key yet: what a part without keys holds is never used, its sum
    a.sum += l;             // is 0, or NaN where every score was
    return;
  }
  const float f = ex2(a.top - next), w = ex2(m - next);
  a.top = next;
  a.sum = a.sum * f + w * l;
  if (w != 0.f) a.o = make_float4(a.o.x * f + w * x.x, a.o.y * f + w * x.y, a.o.z * f + w * x.z, a.o.w * f + w * x.w);
}
// K column groups of a row, U parts' loads at a time.
template <int K, int U>
__device__ __forceinline__ void join_parts(const PagedParams& p, int c, int nparts, int row, int c8, int first, int share,
                                           bool in_row, Joined (&a)[K]) {
#pragma unroll
  for (int k = 0; k < K; ++k) a[k] = Joined{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  for (int i0 = first; i0 < nparts; i0 += U * share) {
    float4 x[U][K];
    float m[U], l[U];
#pragma unroll
    for (int b = 0; b < U; ++b) {
      const int i = i0 + b * share;
      const bool in = in_row && i < nparts;
      const uint8_t* const part = p.parts + (size_t)(i == 0 ? 2 * c + 1 : 2 * (c + i)) * PART_BYTES;
      const float* const ml = reinterpret_cast<const float*>(part + PART_O) + row;
      m[b] = in ? ml[0] : -INFINITY;
      l[b] = in ? ml[256] : 0.f;
#pragma unroll
      for (int k = 0; k < K; ++k)
        x[b][k] = in ? reinterpret_cast<const float4*>(part)[((c8 + 4 * k) * 256 + row) * 2 + (threadIdx.x & 1)]
                     : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int b = 0; b < U; ++b)
#pragma unroll
      for (int k = 0; k < K; ++k) join(a[k], m[b], l[b], x[b][k]);
  }
}
__global__ void __launch_bounds__(COMBINE_THREADS, 4) paged_combine_kernel(const __grid_constant__ PagedParams p) {
  __shared__ Joined s_part[COMBINE_THREADS];
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.y, bx = blockIdx.x;
  const Split s = p.splits[c];
  if (s.last < 0) return;
  const int all = s.ntok * p.G, half0 = min(s.ntok, p.tq) * p.G;  // rows of the work tile, of its first half
  const bool wide = all > 32;
  const int row0 = wide ? bx * 32 : 0, rows = min(32, all - row0);
  if (rows <= 0) return;
  const int nparts = s.last - c + 1, tid = threadIdx.x;
  // Thread number: float4 of a column group (1 bit), row (`shift` bits), column group (2 bits, and
  // three more at distances of 4; or 1 bit), share.
  const int shift = wide || rows > 16 ? 5 : 32 - __clz(rows - 1);  // rows <= 2^shift
  const int r = (tid >> 1) & ((1 << shift) - 1), hi = tid >> (1 + shift);
  const int m = row0 + r, row = m < half0 ? m : 128 + m - half0;
  const int tok = m / p.G;  // row m is token m / G, head m % G
  const long long out_row = (long long)(s.row0 + tok) * p.n_head + s.g * p.G + (m - tok * p.G);
  auto store = [&](const Joined& a, int c8) {
    const float inv = a.sum != 0.f ? 1.0f / a.sum : 0.f;
    reinterpret_cast<uint2*>(p.out + out_row * HD)[c8 * 2 + (tid & 1)] =
        inv != 0.f ? make_uint2(pack_bf16x2(a.o.x * inv, a.o.y * inv), pack_bf16x2(a.o.z * inv, a.o.w * inv))
                   : make_uint2(0, 0);
    if (p.lse && c8 == 0 && (tid & 1) == 0) p.lse[out_row] = a.sum != 0.f ? (a.top + log2f(a.sum)) * LN2 : -INFINITY;
  };
  if (wide) {  // its last rows may be few: the others' threads stay idle
    Joined a[4];
    join_parts<4, 1>(p, c, nparts, row, hi, 0, 1, r < rows, a);
    if (r < rows)
#pragma unroll
      for (int k = 0; k < 4; ++k) store(a[k], hi + 4 * k);
  } else {
    Joined a[1];
    const int first = hi >> 1, share = 64 >> shift;
    join_parts<1, 4>(p, c, nparts, row, 2 * bx + (hi & 1), first, share, r < rows, a);
    s_part[tid] = a[0];
    __syncthreads();
    if (first == 0 && r < rows) {
      for (int i = 1; i < share; ++i) {
        const Joined& y = s_part[tid + i * (4 << shift)];
        join(a[0], y.top, y.sum, y.o);
      }
      store(a[0], 2 * bx + (hi & 1));
    }
  }
}

}  // namespace

size_t paged_attention_scratch_bytes(const moe_paged_shape_t&) { return SCRATCH_BYTES; }

cudaError_t launch_paged_attention(const moe_paged_shape_t& s, const uint16_t* q, long long q_stride,
                                   const uint16_t* k_cache, const uint16_t* v_cache, const int32_t* block_table,
                                   const int32_t* row_start, const int32_t* kv_len, uint16_t* out, float* lse,
                                   void* scratch, cudaStream_t st) {
  PagedParams p;
  std::memset(&p, 0, sizeof(p));
  p.G = s.n_head / s.n_kv_head;
  p.tq = 128;
  while (p.tq * p.G > 128) p.tq >>= 1;  // 128 / (G rounded up to a power of two)
  while ((1 << p.tQ_shift) < 2 * p.tq) ++p.tQ_shift;
  while ((1 << p.page_shift) < s.page_size) ++p.page_shift;
  const uint64_t qdims[4] = {64, 2, (uint64_t)s.n_head, (uint64_t)s.tokens};
  const uint64_t qstrides[3] = {128, 256, (uint64_t)q_stride * 2};
  const uint32_t qbox[4] = {64, 1, (uint32_t)p.G, (uint32_t)p.tq};
  const uint64_t rows = (uint64_t)s.pages * s.n_kv_head * s.page_size;
  const uint64_t kdims[4] = {64, 8, 2, rows / 8}, kstrides[3] = {256, 128, 2048};
  const uint32_t kbox[4] = {64, 8, 2, (uint32_t)s.page_size / 8};
  if (!encode_tma_bf16(&p.q, q, 4, qdims, qstrides, qbox) || !encode_tma_bf16(&p.k, k_cache, 4, kdims, kstrides, kbox) ||
      !encode_tma_bf16(&p.v, v_cache, 4, kdims, kstrides, kbox))
    return cudaErrorInvalidValue;
  p.table = block_table;
  p.row_start = row_start;
  p.kv_len = kv_len;
  p.out = out;
  p.lse = lse;
  p.flags = static_cast<unsigned long long*>(scratch);
  p.splits = reinterpret_cast<Split*>(static_cast<uint8_t*>(scratch) + FLAG_BYTES);
  p.parts = static_cast<uint8_t*>(scratch) + FLAG_BYTES + CTAS * sizeof(Split);
  // An id for every call of the process, from a start that a flag does not hold by chance.  A
  // replay of a captured call has the capture's id and finds the flags cleared.
  static std::atomic<unsigned long long> calls{
      (unsigned long long)std::chrono::steady_clock::now().time_since_epoch().count() << 20 | 1u};
  p.call = calls.fetch_add(1);
  p.status = device_status_ptr();
  if (!p.status) return cudaErrorInvalidDevicePointer;
  p.R = s.requests;
  p.T = s.tokens;
  p.n_head = s.n_head;
  p.n_kv_head = s.n_kv_head;
  p.pages = s.pages;
  p.max_pages = s.max_pages;
  p.scale_log2 = 1.4426950408889634f / sqrtf((float)HD);
  cudaError_t e = cudaFuncSetAttribute(paged_attention_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
  if (e == cudaSuccess) e = launch_pdl(paged_attention_kernel, dim3(CTAS), dim3(THREADS), SMEM_BYTES, st, p);
  if (e == cudaSuccess)
    e = launch_pdl(paged_combine_kernel, dim3(COMBINE_BLOCKS, CTAS), dim3(COMBINE_THREADS), 0, st, p);
  return e;
}

}  // namespace moe
