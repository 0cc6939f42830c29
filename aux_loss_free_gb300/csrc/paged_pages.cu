// Pages of the paged key/value cache between two steps: rows that branch, are cut back or end
// (moe_paged_fork, moe_paged_release), the pages in use moved together (moe_paged_compact), and the
// copies that either asks for (moe_paged_copy) (sm_103a).
//
// The article names no cache: definitions and form are this library's own (moe_gb300.h).
//
// Who holds a page is not kept from call to call: every call reads the tables, marks each page's
// holders in the workspace, and from the marks alone knows which pages are free now, which page with
// room left has more than one holder, and in which order.  Counters kept beside the tables would save
// that pass, but moe_paged_plan, which gives pages out and takes them back, would have to keep them too.
//
// One launch of one cluster: the phases (clear, mark, count, order, write) each need all of the one
// before, a cluster's barrier costs a fraction of a launch, and eight blocks of 1024 threads hold the
// tables of a busy server (a thousand rows of thirty pages) at four entries a thread.  Each block keeps the
// marks of its share of the pages in its shared memory, where the others set them and where it counts
// them without another trip to memory; caches of more than 2^18 pages have theirs in the workspace.  Only
// "holds at all" matters, so marks are byte stores of the same value; the lowest row that ends in a
// page is an atomic maximum, which no order changes.
//
// Bound by latency, a chain of some ten dependent loads and four cluster barriers (1.1k cycles each): 13 rows of up to 128
// pages 7.1 us, 9 rows moved together 6.9 us, 300 rows over 11506 pages 9.0 us; 1021 rows of 33 pages 12.3 us, of which
// the scattered marks (two bytes an entry, to eight blocks) take 6.5 us.  With the marks in the workspace these
// took 9.9, 10.0, 13.9 and 16.6 us; with sixteen blocks 7.6, 7.4, 8.6 and 11.5 us, and two more calls on the host.
// A release marks every page in use whether a row ends or not: 64 rows of up to 16000 tokens 15.8 us in pages of 16
// tokens and 8.9 in pages of 64 (behind a window of 1024, whose pages alone are left, 12.9 and 8.6), 1021 rows of up
// to 900 tokens 20.8 and 9.1 us; the plan behind it takes 3.3 to 5.4 us, both together 12.2 to 29.7.
#include <cuda_bf16.h>

#include <algorithm>

#include "internal.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr unsigned FULL = 0xFFFFFFFFu;
constexpr int HD = kAttnHeadDim;
constexpr int CLUSTER = 8;
constexpr int THREADS = 1024;
constexpr int WARPS = THREADS / 32;
constexpr int ITEM = 64;    // table entries of a row that a warp takes at a time
constexpr int BATCH = 4;    // items whose entries are on their way together
constexpr int GROUP = 16;   // pages that a thread takes at a time: marks in one 16-byte load
constexpr int MARK_BYTES = 6;         // of a page: held before, held as a whole page afterwards, and four for its ends
constexpr int SMEM_SHARE = 1 << 15;   // pages of a block's share, at most, whose marks fit in shared memory

struct PagesParams {
  PagesArgs a;
  uint8_t* marks;   // without shared memory: [CLUSTER][MARK_BYTES << share_shift], as there
  int32_t* length;  // [R] tokens kept
  int32_t* last;    // [R] the page with room left that the row ends in, -1 = none
  int32_t* stage;   // [R][max_pages] new rows, where the table is replaced in place
  int* status;
  int R, pages, max_pages, page_shift;
  int share_shift;  // log2 of the pages of a block's share, at least GROUP
  int in_place;
};

__device__ __forceinline__ int cluster_rank() {
  int r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  cluster_arrive();
  cluster_wait();
}
__device__ __forceinline__ uint32_t in_block(uint32_t smem, int rank) {  // the same place in another block
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem), "r"(rank));
  return r;
}

// The pages' marks: `OLD` held before, `NOW` held as a whole page afterwards (bytes, 0 or 1), and a word: R less
// the lowest row that ends in it, 0 = none (compact: its rank).
template <bool SMEM>
struct Marks {
  uint32_t smem;
  uint8_t* global;
  int shift;  // share_shift
  static constexpr int OLD = 0, NOW = 1;
  __device__ __forceinline__ uint32_t offset(int id, int which) const {
    return (which << shift) + (id & ((1 << shift) - 1));
  }
  __device__ __forceinline__ uint32_t word(int id) const { return (2 << shift) + 4 * (id & ((1 << shift) - 1)); }
  __device__ __forceinline__ uint8_t* share(int rank) const { return global + (size_t)rank * MARK_BYTES * (1u << shift); }
  __device__ __forceinline__ void set(int id, int which) const {
    const int rank = id >> shift;
    if (SMEM) asm volatile("st.shared::cluster.u8 [%0], %1;" ::"r"(in_block(smem, rank) + offset(id, which)), "r"(1) : "memory");
    else share(rank)[offset(id, which)] = 1;
  }
  __device__ __forceinline__ int get(int id, int which) const {
    const int rank = id >> shift;
    uint32_t v;
    if (SMEM) asm volatile("ld.shared::cluster.u8 %0, [%1];" : "=r"(v) : "r"(in_block(smem, rank) + offset(id, which)) : "memory");
    else v = __ldcg(share(rank) + offset(id, which));
    return (int)v;
  }
  __device__ __forceinline__ void raise(int id, int v) const {
    const int rank = id >> shift;
    if (SMEM) asm volatile("red.shared::cluster.max.s32 [%0], %1;" ::"r"(in_block(smem, rank) + word(id)), "r"(v) : "memory");
    else atomicMax(reinterpret_cast<int*>(share(rank) + word(id)), v);
  }
  __device__ __forceinline__ int get_word(int id) const {
    const int rank = id >> shift;
    int v;
    if (SMEM) asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(in_block(smem, rank) + word(id)) : "memory");
    else v = __ldcg(reinterpret_cast<const int*>(share(rank) + word(id)));
    return v;
  }
  // This block's own share.
  __device__ __forceinline__ uint4 load16(int rank, uint32_t at) const {
    uint4 v;
    if (SMEM) asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(smem + at) : "memory");
    else v = __ldcg(reinterpret_cast<const uint4*>(share(rank) + at));
    return v;
  }
  __device__ __forceinline__ void set_word(int rank, int id, int v) const {
    if (SMEM) asm volatile("st.shared.s32 [%0], %1;" ::"r"(smem + word(id)), "r"(v) : "memory");
    else *reinterpret_cast<int*>(share(rank) + word(id)) = v;
  }
  __device__ __forceinline__ void clear(int rank) const {
    for (uint32_t i = threadIdx.x * 16; i < (uint32_t)MARK_BYTES << shift; i += THREADS * 16) {
      if (SMEM) asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(smem + i), "r"(0) : "memory");
      else *reinterpret_cast<uint4*>(share(rank) + i) = make_uint4(0, 0, 0, 0);
    }
  }
  // Of the group of 16 pages `group` of the share, a bit for each page.
  __device__ __forceinline__ uint32_t bits(int rank, int group, int which) const {
    const uint4 v = load16(rank, (which << shift) + GROUP * group);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t b = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)  // each byte is 0 or 1
      b |= ((w[i] * 0x01020408u) >> 24 & 0xFu) << (4 * i);
    return b;
  }
  __device__ __forceinline__ uint32_t ending_bits(int rank, int group) const {
    uint32_t b = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 v = load16(rank, (2 << shift) + 4 * GROUP * group + 16 * i);
      b |= ((v.x != 0) | (v.y != 0) << 1 | (v.z != 0) << 2 | (v.w != 0) << 3) << (4 * i);
    }
    return b;
  }
};

// Sums over the block of two numbers below 2^31.
__device__ __forceinline__ int2 block_sum(int2 v, int2* warp_sums) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  v = make_int2(__reduce_add_sync(FULL, v.x), __reduce_add_sync(FULL, v.y));
  __syncthreads();
  if (lane == 0) warp_sums[warp] = v;
  __syncthreads();
  v = warp_sums[lane];  // 32 warps
  return make_int2(__reduce_add_sync(FULL, v.x), __reduce_add_sync(FULL, v.y));
}
// Exclusive sum over the block; *total the block's.
__device__ __forceinline__ int block_exclusive_sum(int v, int2* warp_sums, int* total) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(FULL, inc, o);
    if (lane >= o) inc += up;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp].x = inc;
  __syncthreads();
  const int mine = warp_sums[lane].x;
  const int before = __reduce_add_sync(FULL, lane < warp ? mine : 0);
  *total = __reduce_add_sync(FULL, mine);
  return before + inc - v;
}
// Every block's sums to every block; read behind the next cluster barrier.
__device__ __forceinline__ void share_sums(int2 v, int2* all, int rank) {
  if (threadIdx.x < CLUSTER)
    asm volatile("st.shared::cluster.v2.s32 [%0], {%1, %2};" ::"r"(in_block(smem_u32(all + rank), threadIdx.x)), "r"(v.x),
                 "r"(v.y)
                 : "memory");
}

__device__ __forceinline__ int pages_of(int tokens, int shift) { return (tokens + (1 << shift) - 1) >> shift; }

// A length within the table (2^24 tokens at most), or 0.
__device__ __forceinline__ int sound_length(const PagesParams& p, int c, bool& bad) {
  if (c >= 0 && c <= p.max_pages << p.page_shift) return c;
  bad = true;
  return 0;
}
__device__ __forceinline__ int sound_page(const PagesParams& p, int id, bool& bad) {
  if (id >= 0 && id < p.pages) return id;
  if (id != -1) bad = true;
  return -1;
}

// The row that row r goes on from, -1 = none, and the tokens that it keeps.
__device__ __forceinline__ int parent_of(const PagesParams& p, int r, bool& bad) {
  if (p.a.new_len) return p.a.new_len[r] < 0 ? -1 : r;
  const int q = p.a.parent ? p.a.parent[r] : r;
  if (q >= -1 && q < p.R) return q;
  bad = true;
  return -1;
}
__device__ __forceinline__ int kept_of(const PagesParams& p, int r, int q, bool& bad) {
  const int keep = p.a.keep ? p.a.keep[r] : 0x7FFFFFFF;
  if (q < 0) return 0;
  return min(max(keep, 0), sound_length(p, p.a.ctx_len[q], bad));
}
// Whether a later token of a row of `len` tokens sees a key of page j.
__device__ __forceinline__ bool seen_again(const PagesParams& p, int j, int len) {
  const int first = j << p.page_shift;
  return p.a.window == 0 || first < p.a.sinks || first + (1 << p.page_shift) > len - p.a.window + 1;
}

// Groups of the block's share of the pages.
__device__ __forceinline__ int groups_of(const PagesParams& p, int rank) {
  const int pages = min(max(p.pages - (rank << p.share_shift), 0), 1 << p.share_shift);
  return (pages + GROUP - 1) / GROUP;
}

// The tables' entries, ITEM of a row at a time, spread over `warps` warps: a lane prepares an item (row, first
// entry, what the others are to know of it; false = nothing there), then the warp takes the lanes' items in
// turn: load gives this lane's entries, of BATCH items before the first use.
template <int N>
struct Entries {
  int v[N][ITEM / 32];
};
// `ready` is called in front of the uses.  An item's info.w: entries of the row, none from there on.
template <int N, class Prepare, class Load, class Ready, class Use>
__device__ __forceinline__ void for_items(const PagesParams& p, int warp, int warps, Prepare prepare, Load load,
                                          Ready ready, Use use) {
  const int lane = threadIdx.x % 32;
  const int per_row = (p.max_pages + ITEM - 1) / ITEM;  // at most 2^14, of 2^12 rows
  const int items = p.R * per_row;
  for (int base = warp; base < items; base += 32 * warps) {
    const int id = base + lane * warps, r = id < items ? id / per_row : 0, c = id < items ? id - r * per_row : 0;
    int4 info = make_int4(0, 0, 0, 0);
    const bool has = id < items && prepare(r, c * ITEM, info);
    for (unsigned left = __ballot_sync(FULL, has); left;) {
      int row[BATCH], first[BATCH];
      int4 about[BATCH];
      Entries<N> e[BATCH];
#pragma unroll
      for (int b = 0; b < BATCH; ++b) {
        row[b] = -1;
        if (!left) continue;
        const int from = __ffs(left) - 1;
        left &= left - 1;
        row[b] = __shfl_sync(FULL, r, from);
        first[b] = __shfl_sync(FULL, c, from) * ITEM + lane;
        about[b] = make_int4(__shfl_sync(FULL, info.x, from), __shfl_sync(FULL, info.y, from),
                             __shfl_sync(FULL, info.z, from), __shfl_sync(FULL, info.w, from));
#pragma unroll
        for (int k = 0; k < ITEM / 32; ++k) load(row[b], first[b] + 32 * k, about[b], e[b], k);
      }
      ready();
#pragma unroll
      for (int b = 0; b < BATCH; ++b) {
        if (row[b] < 0) continue;
#pragma unroll
        for (int k = 0; k < ITEM / 32; ++k)
          if (first[b] - lane + 32 * k < about[b].w) use(row[b], first[b] + 32 * k, about[b], e[b], k);
      }
    }
  }
}

template <bool SMEM>
__global__ void __cluster_dims__(CLUSTER) __launch_bounds__(THREADS, 1)
    paged_fork_kernel(const __grid_constant__ PagesParams p) {
  extern __shared__ __align__(16) uint8_t mark_smem[];
  __shared__ int2 warp_sums[WARPS], sums[CLUSTER];
  const int rank = cluster_rank();
  const int warp = threadIdx.x / 32 * CLUSTER + rank, shift = p.page_shift;  // neighbours in different blocks
  const bool release = p.a.copies == nullptr;
  const Marks<SMEM> marks{smem_u32(mark_smem), p.marks, p.share_shift};
  constexpr int OLD = Marks<SMEM>::OLD, NOW = Marks<SMEM>::NOW;
  bool bad = false;
  if (SMEM) marks.clear(rank);
  pdl_wait();
  pdl_trigger();
  if (!SMEM) marks.clear(rank);
  __syncwarp();
  cluster_arrive();
  bool cleared = false;  // waited for when the first entries are on their way
  auto ready = [&] {
    if (!cleared) cluster_wait();
    cleared = true;
  };

  // ---- marks, and the new rows
  for_items<2>(
      p, warp, CLUSTER * WARPS,
      [&](int r, int j0, int4& info) {
        const int ctx = p.a.ctx_len[r], q = parent_of(p, r, bad), kept = kept_of(p, r, q, bad);
        const int had = pages_of(sound_length(p, ctx, bad), shift);
        info = make_int4(q, had, kept, max(had, pages_of(kept, shift)));
        if (j0 == 0) {
          p.length[r] = kept;
          if (release || (kept & ((1 << shift) - 1)) == 0) p.last[r] = -1;
        }
        return j0 < info.w;
      },
      [&](int r, int j, const int4& info, Entries<2>& e, int k) {  // before, after
        const int q = info.x;
        e.v[0][k] = j < info.y ? p.a.table_in[(long long)r * p.max_pages + j] : -1;
        e.v[1][k] = j < pages_of(info.z, shift) ? q == r ? e.v[0][k] : p.a.table_in[(long long)q * p.max_pages + j] : -1;
      },
      ready,
      [&](int r, int j, const int4& info, const Entries<2>& e, int k) {
        const int q = info.x, kept = info.z, after = e.v[1][k];
        const long long at = (long long)r * p.max_pages + j;
        if (j < info.y) {
          const int id = sound_page(p, e.v[0][k], bad);
          if (id >= 0) marks.set(id, OLD);
        }
        if (j < pages_of(kept, shift)) {
          const int id = seen_again(p, j, kept) ? sound_page(p, after, bad) : -1;
          if (!release && (j + 1) << shift > kept) {
            if (id >= 0) marks.raise(id, p.R - r);
            p.last[r] = id;
          } else {
            if (id >= 0) marks.set(id, NOW);
            if (!p.in_place) p.a.table_out[at] = id;
            else if (q != r) p.stage[at] = id;
            // In place the row's own entries stay, but for one that is no page: that is -1 to every reader
            // already.  What is given up is still a page to the rows that go on from this one; it follows later.
            else if (after < -1 || after >= p.pages) p.a.table_out[at] = -1;
          }
        }
      });
  __syncwarp();
  ready();
  const int head_in = p.a.pool_in[0], count_in = p.a.pool_in[1];
  const bool pool_ok = head_in >= 0 && head_in < p.pages && count_in >= 0 && count_in <= p.pages;
  const int head = pool_ok ? head_in : 0, count = pool_ok ? count_in : 0;
  if (!pool_ok) bad = true;
  auto ring = [&](int place) { return head + place >= p.pages ? head + place - p.pages : head + place; };  // < 2^28
  cluster_sync();

  // ---- pages that nobody holds any more, in the order of their numbers
  const int groups = groups_of(p, rank), first_page = rank << p.share_shift;
  auto freed = [&](int group, int* used) {
    const uint32_t held = marks.bits(rank, group, NOW) | marks.ending_bits(rank, group);
    *used = __popc(held);
    return marks.bits(rank, group, OLD) & ~held;
  };
  int2 found = make_int2(0, 0);  // free, used
  for (int g = threadIdx.x; g < groups; g += THREADS) {
    int used;
    found.x += __popc(freed(g, &used));
    found.y += used;
  }
  // The first block decides which rows want a copy of the page that they end in, `upto` of them before this
  // thread's.
  constexpr int MOST = kPagedMaxRequests / THREADS;  // rows of a thread, at most
  const int per = (p.R + THREADS - 1) / THREADS;
  const int r0 = min(p.R, (int)threadIdx.x * per), r1 = min(p.R, r0 + per);
  int last[MOST], kept[MOST], upto = 0, all_wants = 0;
  uint32_t want = 0;
  if (rank == 0) {
#pragma unroll
    for (int i = 0; i < MOST; ++i) {
      kept[i] = r0 + i < r1 ? __ldcg(p.length + r0 + i) : 0;
      last[i] = r0 + i < r1 ? __ldcg(p.last + r0 + i) : -1;
    }
#pragma unroll
    for (int i = 0; i < MOST; ++i)
      if (last[i] >= 0 && (marks.get(last[i], NOW) != 0 || marks.get_word(last[i]) != p.R - (r0 + i))) want |= 1u << i;
    upto = block_exclusive_sum(__popc(want), warp_sums, &all_wants);
  }
  share_sums(block_sum(found, warp_sums), sums, rank);
  cluster_sync();
  int place = 0, all_free = 0, all_used = 0;
#pragma unroll
  for (int c = 0; c < CLUSTER; ++c) {
    if (c < rank) place += sums[c].x;
    all_free += sums[c].x;
    all_used += sums[c].y;
  }
  if (count + all_free > p.pages) bad = true;
  for (int g0 = 0; g0 < groups; g0 += THREADS) {
    const int g = g0 + threadIdx.x;
    int used, total;
    uint32_t bits = g < groups ? freed(g, &used) : 0u;
    int k = place + block_exclusive_sum(__popc(bits), warp_sums, &total);
    for (; bits; bits &= bits - 1, ++k)
      if (k < p.pages - count) p.a.pool[ring(count + k)] = first_page + g * GROUP + __ffs(bits) - 1;
    place += total;
  }
  cluster_sync();

  if (rank != 0) {
    // ---- in place: the new rows over the old, but for the pages with room left
    if (p.in_place) {
      for_items<1>(
          p, threadIdx.x / 32 * (CLUSTER - 1) + rank - 1, (CLUSTER - 1) * WARPS,
          [&](int r, int j0, int4& info) {
            bool ignored = false;
            const int kept = __ldcg(p.length + r), q = parent_of(p, r, ignored);
            // Pages written: all whole ones of another row's, what was given up of its own.
            info = make_int4(q == r, kept, 0, release ? pages_of(kept, shift) : kept >> shift);
            return j0 < info.w && (q != r || p.a.window > 0);
          },
          [&](int r, int j, const int4& info, Entries<1>& e, int k) {
            e.v[0][k] = j < info.w && !info.x ? __ldcg(p.stage + (long long)r * p.max_pages + j) : -1;
          },
          [] {},
          [&](int r, int j, const int4& info, const Entries<1>& e, int k) {
            if (j < info.w && (!info.x || !seen_again(p, j, info.y))) p.a.table_out[(long long)r * p.max_pages + j] = e.v[0][k];
          });
    }
  } else {
    // ---- the rows' lengths and their pages with room left
    const int avail = min(count + all_free, p.pages);
    const int taken = min(all_wants, avail);
#pragma unroll
    for (int i = 0; i < MOST; ++i) {
      const int r = r0 + i;
      if (r >= r1) break;
      const int room = kept[i] & ((1 << shift) - 1);
      if (!release && room) {
        int32_t* const entry = p.a.table_out + (long long)r * p.max_pages + (kept[i] >> shift);
        if (!(want >> i & 1)) {
          *entry = last[i];
        } else if (upto < avail) {
          const int id = __ldcg(p.a.pool + ring(upto));
          if (id < 0 || id >= p.pages) bad = true;
          *entry = id;
          reinterpret_cast<int4*>(p.a.copies)[upto++] = make_int4(last[i], id, room, 0);
        } else {
          ++upto;
          kept[i] -= room;
        }
      }
      p.a.next_ctx[r] = kept[i];
    }
    if (threadIdx.x == 0) {
      p.a.pool_out[0] = ring(taken);
      p.a.pool_out[1] = avail - taken;
      p.a.info[0] = taken;
      p.a.info[1] = all_free;
      p.a.info[2] = all_wants - taken;
      p.a.info[3] = all_used + taken;
    }
  }
  if (bad) atomicOr(p.status, kDevCheck);
}

// The pages in use to [0, n).  With c(x) the pages in use below x, the k-th unused page x below n is
// x - c(x) = k, and the k-th in use from n on is c(x) - c(n) = k: one prefix sum over the marks.
template <bool SMEM>
__global__ void __cluster_dims__(CLUSTER) __launch_bounds__(THREADS, 1)
    paged_compact_kernel(const __grid_constant__ PagesParams p) {
  extern __shared__ __align__(16) uint8_t mark_smem[];
  __shared__ int2 warp_sums[WARPS], sums[CLUSTER], below_n[CLUSTER];
  const int rank = cluster_rank();
  const int warp = threadIdx.x / 32 * CLUSTER + rank, shift = p.page_shift;
  const Marks<SMEM> marks{smem_u32(mark_smem), p.marks, p.share_shift};
  constexpr int NOW = Marks<SMEM>::NOW;
  int4* const copies = reinterpret_cast<int4*>(p.a.copies);
  bool bad = false;
  if (SMEM) marks.clear(rank);
  pdl_wait();
  pdl_trigger();
  if (!SMEM) marks.clear(rank);
  __syncwarp();
  cluster_arrive();
  bool cleared = false;  // waited for when the first entries are on their way
  auto ready = [&] {
    if (!cleared) cluster_wait();
    cleared = true;
  };
  auto rows = [&](auto&& each) {  // each(entry's place, what it holds)
    for_items<1>(
        p, warp, CLUSTER * WARPS,
        [&](int r, int j0, int4& info) {
          info.w = pages_of(sound_length(p, p.a.ctx_len[r], bad), shift);
          return j0 < info.w;
        },
        [&](int r, int j, const int4& info, Entries<1>& e, int k) {
          e.v[0][k] = j < info.w ? p.a.table_in[(long long)r * p.max_pages + j] : -1;
        },
        ready,
        [&](int r, int j, const int4& info, const Entries<1>& e, int k) {
          if (j < info.w) each((long long)r * p.max_pages + j, sound_page(p, e.v[0][k], bad));
        });
  };
  rows([&](long long, int id) {
    if (id >= 0) marks.set(id, NOW);
  });
  __syncwarp();
  ready();
  cluster_sync();

  const int groups = groups_of(p, rank), first_page = rank << p.share_shift;
  int2 found = make_int2(0, 0);
  for (int g = threadIdx.x; g < groups; g += THREADS) found.x += __popc(marks.bits(rank, g, NOW));
  share_sums(block_sum(found, warp_sums), sums, rank);
  cluster_sync();
  int below = 0, n = 0;  // pages in use before the block's share, and all of them
#pragma unroll
  for (int c = 0; c < CLUSTER; ++c) {
    if (c < rank) below += sums[c].x;
    n += sums[c].x;
  }
  __shared__ int found_n;  // pages in use among the first n, if page n lies in this share
  if (threadIdx.x == 0) found_n = -1;
  __syncthreads();
  for (int g0 = 0; g0 < groups; g0 += THREADS) {
    const int g = g0 + threadIdx.x, first = first_page + g * GROUP;
    const uint32_t bits = g < groups ? marks.bits(rank, g, NOW) : 0u;
    int all;
    const int c0 = below + block_exclusive_sum(__popc(bits), warp_sums, &all);  // c(first)
    if (g < groups) {
      if (first <= n && n < first + GROUP) found_n = c0 + __popc(bits & ((1u << (n - first)) - 1u));
#pragma unroll 1
      for (int i = 0; i < GROUP && first + i < p.pages; ++i) {
        const int x = first + i, c = c0 + __popc(bits & ((1u << i) - 1u));
        if (x < n && !(bits >> i & 1)) copies[x - c].y = x;
        if (x >= n && (bits >> i & 1)) marks.set_word(rank, x, c);
      }
    }
    below += all;
  }
  __syncthreads();
  share_sums(make_int2(found_n, 0), below_n, rank);
  cluster_sync();
  int c_n = -1;
#pragma unroll
  for (int c = 0; c < CLUSTER; ++c) c_n = max(c_n, below_n[c].x);
  if (c_n < 0) c_n = n;  // page n lies behind the last one
  const int moves = n - c_n;
  for (int g = threadIdx.x; g < groups; g += THREADS) {
    const int first = first_page + g * GROUP;
    if (first + GROUP <= n) continue;
    for (uint32_t bits = marks.bits(rank, g, NOW); bits; bits &= bits - 1) {
      const int x = first + __ffs(bits) - 1;
      if (x < n) continue;
      int4* const job = copies + (marks.get_word(x) - c_n);
      job->x = x;
      *reinterpret_cast<int2*>(&job->z) = make_int2(1 << shift, 0);
    }
  }
  rows([&](long long at, int id) {
    p.a.table_out[at] = id >= n ? __ldcg(&copies[marks.get_word(id) - c_n].y) : id;
  });
  __syncwarp();
  cluster_arrive();  // the other blocks' marks are read
  for (int k = rank * THREADS + threadIdx.x; k < p.pages - n; k += CLUSTER * THREADS) p.a.pool[k] = n + k;
  if (rank == 0 && threadIdx.x == 0) {
    p.a.pool_out[0] = 0;
    p.a.pool_out[1] = p.pages - n;
    p.a.info[0] = moves;
    p.a.info[1] = 0;
    p.a.info[2] = 0;
    p.a.info[3] = n;
  }
  if (bad) atomicOr(p.status, kDevCheck);
  __syncwarp();
  cluster_wait();  // no block's shared memory goes before it has been read
}

// A warp takes sixteen tokens of one head of one cache: 4 KB, every lane's eight loads on their way
// before the first store.  Bound by memory traffic: 2136 pages of 64 tokens in four caches (560 MB) 87 us, 6.4 TB/s.
constexpr int COPY_CACHES = 64;
constexpr int COPY_TOKENS = 16;
constexpr int COPY_THREADS = 256;
struct CopyParams {
  const int4* copies;
  const int32_t* n_copies;
  uint16_t* caches[COPY_CACHES];
  int* status;
  int n_caches, max_copies, n_kv_head, pages, page_shift;
};
__global__ void __launch_bounds__(COPY_THREADS) paged_copy_kernel(const __grid_constant__ CopyParams p) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x % 32;
  const int n = min(max(*p.n_copies, 0), p.max_copies);
  const int pieces = 1 << (p.page_shift - 4);
  const long long per_copy = (long long)p.n_caches * p.n_kv_head * pieces, items = n * per_copy;
  const long long warps = (long long)gridDim.x * (COPY_THREADS / 32);
  bool bad = false;
  for (long long it = (long long)blockIdx.x * (COPY_THREADS / 32) + threadIdx.x / 32; it < items; it += warps) {
    const int i = (int)(it / per_copy), rest = (int)(it - i * per_copy);
    const int piece = rest & (pieces - 1), which = rest >> (p.page_shift - 4);
    const int g = which % p.n_kv_head;
    const int4 job = p.copies[i];
    if (job.x < 0 || job.x >= p.pages || job.y < 0 || job.y >= p.pages || job.z < 0 || job.z > 1 << p.page_shift) {
      bad = true;
      continue;
    }
    const int vecs = (min(job.z, (piece + 1) * COPY_TOKENS) - piece * COPY_TOKENS) * (HD / 8);
    uint16_t* const cache = p.caches[which / p.n_kv_head];
    auto at = [&](int page) {
      return reinterpret_cast<uint4*>(
          cache + ((((long long)page * p.n_kv_head + g) << p.page_shift) + piece * COPY_TOKENS) * HD);
    };
    const uint4* const src = at(job.x);
    uint4* const dst = at(job.y);
    uint4 v[COPY_TOKENS * (HD / 8) / 32];
#pragma unroll
    for (int k = 0; k < COPY_TOKENS * (HD / 8) / 32; ++k)
      if (32 * k + lane < vecs) v[k] = src[32 * k + lane];
#pragma unroll
    for (int k = 0; k < COPY_TOKENS * (HD / 8) / 32; ++k)
      if (32 * k + lane < vecs) dst[32 * k + lane] = v[k];
  }
  if (bad) atomicOr(p.status, kDevCheck);
}

size_t up16(size_t n) { return (n + 15) / 16 * 16; }

// log2 of the pages of a block's share.
int share_shift_of(const moe_paged_shape_t& s) {
  int shift = 4;
  while ((long long)CLUSTER << shift < s.pages) ++shift;
  return shift;
}
bool marks_in_smem(const moe_paged_shape_t& s) { return 1 << share_shift_of(s) <= SMEM_SHARE; }

struct PagesWs {
  size_t marks, length, last, stage, bytes;
};
PagesWs pages_ws(const moe_paged_shape_t& s) {
  const size_t R = up16(sizeof(int32_t) * (size_t)s.requests);
  PagesWs w;
  w.marks = 0;
  w.length = w.marks + (marks_in_smem(s) ? 0 : (size_t)CLUSTER * MARK_BYTES << share_shift_of(s));
  w.last = w.length + R;
  w.stage = w.last + R;
  w.bytes = w.stage + up16(sizeof(int32_t) * (size_t)s.requests * s.max_pages);
  return w;
}

cudaError_t launch_pages(void (*smem_kernel)(PagesParams), void (*global_kernel)(PagesParams), const moe_paged_shape_t& s,
                         const PagesArgs& a, void* scratch, cudaStream_t st) {
  const PagesWs w = pages_ws(s);
  uint8_t* const base = static_cast<uint8_t*>(scratch);
  PagesParams p{};
  p.a = a;
  p.marks = base + w.marks;
  p.length = reinterpret_cast<int32_t*>(base + w.length);
  p.last = reinterpret_cast<int32_t*>(base + w.last);
  p.stage = reinterpret_cast<int32_t*>(base + w.stage);
  p.status = device_status_ptr();
  if (!p.status) return cudaErrorInvalidDevicePointer;
  p.R = s.requests;
  p.pages = s.pages;
  p.max_pages = s.max_pages;
  while ((1 << p.page_shift) < s.page_size) ++p.page_shift;
  p.share_shift = share_shift_of(s);
  p.in_place = a.table_in == a.table_out;
  if (!marks_in_smem(s)) return launch_pdl(global_kernel, dim3(CLUSTER), dim3(THREADS), 0, st, p);
  const size_t smem = (size_t)MARK_BYTES << p.share_shift;
  if (smem > 40 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(smem_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, MARK_BYTES * SMEM_SHARE);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(smem_kernel, dim3(CLUSTER), dim3(THREADS), smem, st, p);
}

}  // namespace

size_t paged_pages_scratch_bytes(const moe_paged_shape_t& s) { return pages_ws(s).bytes; }

cudaError_t launch_paged_fork(const moe_paged_shape_t& s, const PagesArgs& a, void* scratch, cudaStream_t st) {
  return launch_pages(paged_fork_kernel<true>, paged_fork_kernel<false>, s, a, scratch, st);
}

cudaError_t launch_paged_compact(const moe_paged_shape_t& s, const PagesArgs& a, void* scratch, cudaStream_t st) {
  return launch_pages(paged_compact_kernel<true>, paged_compact_kernel<false>, s, a, scratch, st);
}

cudaError_t launch_paged_copy(const moe_paged_shape_t& s, const int32_t* copies, const int32_t* n_copies, int max_copies,
                              int n_caches, void* const* caches, cudaStream_t st) {
  CopyParams p{};
  p.copies = reinterpret_cast<const int4*>(copies);
  p.n_copies = n_copies;
  p.status = device_status_ptr();
  if (!p.status) return cudaErrorInvalidDevicePointer;
  p.max_copies = max_copies;
  p.n_kv_head = s.n_kv_head;
  p.pages = s.pages;
  while ((1 << p.page_shift) < s.page_size) ++p.page_shift;
  for (int c0 = 0; c0 < n_caches && max_copies > 0; c0 += COPY_CACHES) {
    p.n_caches = std::min(COPY_CACHES, n_caches - c0);
    for (int i = 0; i < p.n_caches; ++i) p.caches[i] = static_cast<uint16_t*>(caches[c0 + i]);
    const long long items = (long long)max_copies * p.n_caches * s.n_kv_head * (s.page_size / COPY_TOKENS);
    const long long blocks = (items + COPY_THREADS / 32 - 1) / (COPY_THREADS / 32);
    const cudaError_t e = launch_pdl(paged_copy_kernel, dim3((unsigned)std::min<long long>(blocks, 152 * 8)),
                                     dim3(COPY_THREADS), 0, st, p);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace moe
