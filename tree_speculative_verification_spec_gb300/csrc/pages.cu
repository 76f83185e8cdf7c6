// Page calls of the paged K/V cache: fork rows of the block table, free rows,
// and compact the pool.
//
// The block table is the only record of who holds a page: a page is held by
// every row that names it, free when the pool lists it, and neither otherwise
// (the caller keeps it for itself).  No counter has to be kept in step with
// the commit's page release, which hands tree pages back by the table alone.
//
// Each call is a plan on the table and the pool (small integer arrays) and,
// for fork and compact, one grid-wide copy of the rows or pages that the plan
// lists, in every layer.  Pool order is fixed by the arguments alone: the
// atomics below are integer minima and counts, and positions come from scans.
// The plans are bound by the latency of their few dependent passes (a free of
// 64 rows of a 256 x 1024 table: 16 + 4 + 15 us for check, mark and release),
// the copies by HBM: 600 pages of 2 MB move at 6.4 TB/s, the partial pages of
// 64 forks (32 layers, pages of 256 slots) at 6.5 TB/s.
#include <algorithm>

#include <cooperative_groups.h>

#include "common.cuh"

namespace cg = cooperative_groups;

namespace spectree {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPlanCluster = 8;
constexpr int kScanThreads = 256;  // grid-wide passes over the table

// A call's kernels are programmatic dependents of one another: each but the last
// lets the next one launch as it starts, and each but the first begins by waiting
// for the one before (its whole grid, results included).
__device__ __forceinline__ void let_next_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_last() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Move of `rows` slots (all of a page, or its first ones) from page src to
// page dst.
struct PageMove {
  int src, dst, rows;
};

// Exclusive prefix (and total) of one value per thread over the cluster, in
// rank-major thread order.  Every thread of every CTA calls it.
struct ClusterScan {
  long long warp[kPlanWarps];
  long long cta[kPlanCluster];
};
__device__ __forceinline__ long long cluster_scan(cg::cluster_group& cl, ClusterScan& sh, long long v,
                                                  long long& total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  long long incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) sh.warp[w] = incl;
  __syncthreads();
  if (w == 0) {
    long long x = sh.warp[lane], xi = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, xi, o);
      if (lane >= o) xi += y;
    }
    sh.warp[lane] = xi - x;
    const long long all = __shfl_sync(0xffffffffu, xi, 31);
    if (lane < C) cl.map_shared_rank(&sh, lane)->cta[rank] = all;
  }
  cl.sync();
  long long base = sh.warp[w] + incl - v;
  total = 0;
  for (int r = 0; r < C; ++r) {
    base += r < rank ? sh.cta[r] : 0;
    total += sh.cta[r];
  }
  cl.sync();  // sh is read everywhere before a later scan writes it
  return base;
}

// ---------------------------------------------------------------------------
// Copy of the listed moves, every layer's K and V cache
// ---------------------------------------------------------------------------
// Cache c is layer c / 2's K (even) or V (odd).  The unit of work is one
// kMoveBytes piece of one head's rows of one page in one cache: contiguous at
// both ends, one warp's 16-byte loads all in flight before its stores.
// Sources are never destinations, so units are independent.
constexpr int kMoveVec = 8;                      // 16-byte vectors per lane
constexpr int kMoveBytes = kMoveVec * 32 * 16;   // 4 KB
constexpr int kMoveThreads = 256;
constexpr int kMoveCtas = 16;                    // per SM; four fit at once: the later ones even out the end
                                                 // (600 pages: 408 us with 4, 404 with 8, 398 with 16 on a cold GPU)

// The plan's results come by plain pointers: a read-only load could be moved
// before the wait.
__global__ void __launch_bounds__(kMoveThreads) page_move_kernel(char* const* k_caches, char* const* v_caches, int n_caches,
                                                                 const PageMove* moves, const int* n_moves, int Hkv,
                                                                 long long head_bytes, int row_bytes, int whole,
                                                                 int32_t* table, long long entries,
                                                                 const int32_t* page_map, int num_blocks) {
  const int lane = threadIdx.x & 31;
  wait_for_last();
  // compaction: the table's entries take their pages' new ids
  for (long long e = (long long)blockIdx.x * kMoveThreads + threadIdx.x; e < entries;
       e += (long long)gridDim.x * kMoveThreads) {
    const int p = table[e];
    if (p >= 0 && p < num_blocks) {
      const int q = page_map[p];
      if (q != p) table[e] = q;
    }
  }
  const long long warps = (long long)gridDim.x * (kMoveThreads / 32);
  // whole pages: the heads of a page lie one after another, one span of all of them
  const int spans = whole ? 1 : Hkv;
  const long long span_bytes = whole ? Hkv * head_bytes : head_bytes;
  const long long pieces = (span_bytes + kMoveBytes - 1) / kMoveBytes;
  const long long units = (long long)*n_moves * n_caches * spans * pieces;
  for (long long u = (long long)blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5); u < units; u += warps) {
    const long long piece = u % pieces;
    long long r = u / pieces;
    const int h = (int)(r % spans);
    r /= spans;
    const int c = (int)(r % n_caches);
    const PageMove m = moves[r / n_caches];
    const long long bytes = whole ? span_bytes : (long long)m.rows * row_bytes;
    const long long at = piece * kMoveBytes;
    if (at >= bytes) continue;
    char* cache = (c & 1) ? v_caches[c >> 1] : k_caches[c >> 1];
    const long long page_bytes = Hkv * head_bytes;
    const uint4* from = reinterpret_cast<const uint4*>(cache + m.src * page_bytes + h * head_bytes + at);
    uint4* to = reinterpret_cast<uint4*>(cache + m.dst * page_bytes + h * head_bytes + at);
    const int n = (int)(min((long long)kMoveBytes, bytes - at) / 16);
    uint4 v[kMoveVec];
#pragma unroll
    for (int i = 0; i < kMoveVec; ++i)
      if (i * 32 + lane < n) v[i] = from[i * 32 + lane];
#pragma unroll
    for (int i = 0; i < kMoveVec; ++i)
      if (i * 32 + lane < n) to[i * 32 + lane] = v[i];
  }
}

// ---------------------------------------------------------------------------
// Fork
// ---------------------------------------------------------------------------
struct ForkArgs {
  int32_t* table;
  const int32_t *src, *dst, *len, *room;
  int32_t *pool, *count, *status;
  int* mark;        // [B] how often a row is a destination
  long long* need;  // [N] fresh pages before fork i; -1: not done
  PageMove* moves;  // [N]
  int* n_moves;
  int B, max_blocks, bs, num_blocks, N, pool_cap;
  int copies;  // a copying kernel follows
};

// One cluster.  Fork i is checked by one warp; fresh pages are numbered by a
// scan over the forks, so fork i takes pool[count - 1 - need[i] - t], t = 0...
__global__ void __launch_bounds__(kPlanThreads) pages_fork_kernel(const ForkArgs a) {
  __shared__ ClusterScan scan;
  __shared__ int s_badpool;
  cg::cluster_group cl = cg::this_cluster();
  if (a.copies) let_next_launch();  // else the next kernel is not this call's
  const int G = (int)cl.num_blocks() * kPlanThreads, id = (int)cl.block_rank() * kPlanThreads + threadIdx.x;
  const int lane = threadIdx.x & 31;
  const int warps = G / 32, wid = id / 32;
  if (threadIdx.x == 0) s_badpool = 0;
  for (int i = id; i < a.N; i += G) {
    const int s = a.src[i], d = a.dst[i];
    if (s >= 0 && s < a.B) a.mark[s] = 0;
    if (d >= 0 && d < a.B) a.mark[d] = 0;
  }
  __threadfence();
  cl.sync();
  for (int i = id; i < a.N; i += G)
    if (a.dst[i] >= 0 && a.dst[i] < a.B) atomicAdd(&a.mark[a.dst[i]], 1);
  __threadfence();
  cl.sync();
  // checks, and the number of fresh pages
  for (int i = wid; i < a.N; i += warps) {
    const int s = a.src[i], d = a.dst[i], len = a.len[i], room = a.room ? a.room[i] : 0;
    int bad = 0, fresh = 0;
    if (s < -1 || s >= a.B || d < 0 || d >= a.B || len < 0 || room < 0 || (s < 0 && len > 0)) bad = SPEC_DEV_BAD_ROW;
    else if (__ldcg(&a.mark[d]) != 1 || (s >= 0 && s != d && __ldcg(&a.mark[s]) != 0)) bad = SPEC_DEV_BAD_ROW;
    else if ((long long)len + room > (long long)a.max_blocks * a.bs) bad = SPEC_DEV_CAPACITY;
    if (!bad) {
      const int full = len / a.bs, held = (int)(((long long)len + a.bs - 1) / a.bs), need = (int)(((long long)len + room + a.bs - 1) / a.bs);
      const int32_t* drow = a.table + (size_t)d * a.max_blocks;
      const int32_t* srow = s >= 0 ? a.table + (size_t)s * a.max_blocks : drow;
      int bad_id = 0, taken = 0;
      for (int j = lane; j < max(held, need); j += 32) {
        if (j < held) bad_id |= srow[j] < 0 || srow[j] >= a.num_blocks;
        if (s == d) {
          if (j >= held && j < need) {
            fresh += drow[j] < 0;
            bad_id |= drow[j] >= a.num_blocks;
          }
        } else {
          taken |= drow[j] >= 0;
          fresh += j >= full;
        }
      }
      if (__any_sync(0xffffffffu, bad_id)) bad |= SPEC_DEV_BAD_BLOCK;
      if (__any_sync(0xffffffffu, taken)) bad |= SPEC_DEV_BAD_ROW;
      fresh = warp_sum_i(fresh);
    }
    if (lane == 0) {
      a.status[i] = bad;
      a.need[i] = bad ? -1 : fresh;
      a.moves[i] = PageMove{0, 0, 0};
    }
  }
  __threadfence();
  cl.sync();
  // where each fork's fresh pages start: thread `id` owns a run of forks
  const int per = (a.N + G - 1) / G;
  const int i0 = min(a.N, id * per), i1 = min(a.N, i0 + per);
  long long mine = 0, total = 0;
  for (int i = i0; i < i1; ++i) mine += max(0LL, __ldcg(&a.need[i]));
  long long at = cluster_scan(cl, scan, mine, total);
  const int count = *(volatile int32_t*)a.count;
  int short_of = 0;
  if (total > 0 && (count < 0 || count > a.pool_cap || total > count)) {
    short_of = SPEC_DEV_CAPACITY;
  } else {  // the ids that are about to be handed out
    int b = 0;
    for (long long t = id; t < total; t += G) {
      const int p = a.pool[count - 1 - t];
      b |= p < 0 || p >= a.num_blocks;
    }
    if (__syncthreads_or(b) && threadIdx.x < cl.num_blocks()) *cl.map_shared_rank(&s_badpool, threadIdx.x) = 1;
  }
  cl.sync();
  if (s_badpool) short_of = SPEC_DEV_BAD_BLOCK;
  for (int i = i0; i < i1; ++i) {
    const long long n = __ldcg(&a.need[i]);
    if (n > 0 && short_of) {
      a.status[i] = short_of;
      a.need[i] = -1;
    } else if (n >= 0) {
      a.need[i] = at;
      at += n;
    }
  }
  __threadfence();
  cl.sync();
  // the new rows
  for (int i = wid; i < a.N; i += warps) {
    const long long first = __ldcg(&a.need[i]);
    if (first < 0) continue;
    const int s = a.src[i], d = a.dst[i], len = a.len[i], room = a.room ? a.room[i] : 0;
    const int full = len / a.bs, held = (int)(((long long)len + a.bs - 1) / a.bs), need = (int)(((long long)len + room + a.bs - 1) / a.bs);
    int32_t* drow = a.table + (size_t)d * a.max_blocks;
    if (s == d) {
      int nth = 0;
      for (int j0 = held; j0 < need; j0 += 32) {
        const int j = j0 + lane;
        const bool empty = j < need && drow[j] < 0;
        const unsigned m = __ballot_sync(0xffffffffu, empty);
        if (empty) drow[j] = a.pool[count - 1 - (first + nth + __popc(m & ((1u << lane) - 1u)))];
        nth += __popc(m);
      }
    } else {
      const int32_t* srow = s >= 0 ? a.table + (size_t)s * a.max_blocks : nullptr;
      for (int j = lane; j < need; j += 32)
        drow[j] = j < full ? srow[j] : a.pool[count - 1 - (first + (j - full))];
      if (lane == 0 && len > full * a.bs) a.moves[i] = PageMove{srow[full], a.pool[count - 1 - first], len - full * a.bs};
    }
  }
  cl.sync();  // every read of the pool precedes the new count
  if (id == 0) {
    if (!short_of) *a.count = count - (int)total;
    *a.n_moves = a.N;
  }
}

// ---------------------------------------------------------------------------
// Free
// ---------------------------------------------------------------------------
struct FreeArgs {
  int32_t* table;
  const int32_t *rows, *keep;
  int32_t *pool, *count, *status;
  int *from;   // [B] first dropped page of a row (max_blocks: none)
  int *entry;  // [B] the entry that drops it
  int *mark;   // [B]
  int *first;  // [num_blocks] first position that drops a page, -1 when a row keeps it
  int B, max_blocks, bs, num_blocks, N, pool_cap;
};

// One cluster: which entries are sound, and the pages they would drop.
__global__ void __launch_bounds__(kPlanThreads) pages_free_check_kernel(const FreeArgs a) {
  cg::cluster_group cl = cg::this_cluster();
  let_next_launch();
  const int G = (int)cl.num_blocks() * kPlanThreads, id = (int)cl.block_rank() * kPlanThreads + threadIdx.x;
  for (int r = id; r < a.B; r += G) {
    a.from[r] = a.max_blocks;
    a.mark[r] = 0;
  }
  __threadfence();
  cl.sync();
  for (int i = id; i < a.N; i += G)
    if (a.rows[i] >= 0 && a.rows[i] < a.B) atomicAdd(&a.mark[a.rows[i]], 1);
  __threadfence();
  cl.sync();
  for (int i = id; i < a.N; i += G) {
    const int r = a.rows[i], keep = a.keep ? a.keep[i] : 0;
    const bool sound = r >= 0 && r < a.B && keep >= 0 && __ldcg(&a.mark[r]) == 1;
    a.status[i] = sound ? 0 : SPEC_DEV_BAD_ROW;
    if (sound) {
      a.from[r] = (int)min((long long)a.max_blocks, ((long long)keep + a.bs - 1) / a.bs);
      a.entry[r] = i;
    }
  }
  __threadfence();
  cl.sync();
  // The pages they would drop start as "dropped by no position" (one listed in
  // a row found bad here is never looked up).  Eight entries are loaded before
  // any is used: row by row and one by one this took 26 us on 64 rows of 1024.
  constexpr int kAt = 8;
  const long long n = (long long)a.N * a.max_blocks;
  for (long long e0 = id; e0 < n; e0 += (long long)kAt * G) {
    int p[kAt], i[kAt];
#pragma unroll
    for (int q = 0; q < kAt; ++q) {
      const long long e = e0 + (long long)q * G;
      i[q] = e < n ? (int)(e / a.max_blocks) : -1;
      p[q] = -1;
      if (i[q] >= 0 && __ldcg(&a.status[i[q]]) != SPEC_DEV_BAD_ROW) {
        const int r = a.rows[i[q]], j = (int)(e - (long long)i[q] * a.max_blocks);
        if (j >= __ldcg(&a.from[r])) p[q] = a.table[(size_t)r * a.max_blocks + j];
      }
    }
#pragma unroll
    for (int q = 0; q < kAt; ++q) {
      if (p[q] >= a.num_blocks) atomicOr(&a.status[i[q]], SPEC_DEV_BAD_BLOCK);
      else if (p[q] >= 0) a.first[p[q]] = INT32_MAX;
    }
  }
  __threadfence();
  cl.sync();
  for (int i = id; i < a.N; i += G)
    if (__ldcg(&a.status[i]) & SPEC_DEV_BAD_BLOCK) a.from[a.rows[i]] = a.max_blocks;
}

// Every entry of the table: a page a row keeps is marked -1, a dropped one
// with its lowest position (entry, then page).
__global__ void __launch_bounds__(kScanThreads) pages_free_mark_kernel(const FreeArgs a) {
  let_next_launch();
  wait_for_last();
  const int chunks = (a.max_blocks + kScanThreads - 1) / kScanThreads;  // a CTA takes one row's chunk at a time
  for (int u = blockIdx.x; u < a.B * chunks; u += gridDim.x) {
    const int r = u / chunks, j = (u - r * chunks) * kScanThreads + threadIdx.x;
    if (j >= a.max_blocks) continue;
    const int p = a.table[(size_t)r * a.max_blocks + j];
    if (p >= 0 && p < a.num_blocks)
      atomicMin(&a.first[p], j < a.from[r] ? -1 : a.entry[r] * a.max_blocks + j);
  }
}

// One cluster: the released pages go to the pool in position order, the
// dropped entries become -1.
__global__ void __launch_bounds__(kPlanThreads) pages_free_release_kernel(const FreeArgs a) {
  __shared__ ClusterScan scan;
  cg::cluster_group cl = cg::this_cluster();
  const int G = (int)cl.num_blocks() * kPlanThreads, id = (int)cl.block_rank() * kPlanThreads + threadIdx.x;
  cl.sync();  // every CTA runs: the scan writes to the others' shared memory
  wait_for_last();
  const int n = a.N * a.max_blocks;  // at most 2^30
  const int count = *(volatile int32_t*)a.count;
  // Thread `id` owns a run of positions (one scan for the call), eight of them
  // looked up at a time, since each is a chain of four loads.
  constexpr int kAt = 8;
  const int per = (int)(((long long)n + G - 1) / G);
  const int e0 = (int)min((long long)n, (long long)id * per), e1 = (int)min((long long)n, (long long)e0 + per);
  int32_t* at[kAt];  // the table entry that position e + q drops, or NULL
  int page[kAt];
  unsigned out = 0;  // which of them release their page
  auto look = [&](int e) {
    out = 0;
#pragma unroll
    for (int q = 0; q < kAt; ++q) {
      at[q] = nullptr;
      page[q] = -1;
      if (e + q < e1) {
        const int i = (e + q) / a.max_blocks, j = e + q - i * a.max_blocks;
        const int st = a.status[i], r = a.rows[i];
        if ((st & (SPEC_DEV_BAD_ROW | SPEC_DEV_BAD_BLOCK)) == 0 && j >= a.from[r]) {
          at[q] = a.table + (size_t)r * a.max_blocks + j;
          page[q] = *at[q];
        }
      }
    }
#pragma unroll
    for (int q = 0; q < kAt; ++q)
      if (page[q] >= 0 && a.first[page[q]] == e + q) out |= 1u << q;
  };
  int mine = 0;
  for (int e = e0; e < e1; e += kAt) {
    look(e);
    mine += __popc(out);
  }
  long long total = 0;
  long long pos = count + cluster_scan(cl, scan, mine, total);
  const bool fits = total == 0 || (count >= 0 && count + total <= a.pool_cap);
  for (int e = e0; e < e1; e += kAt) {
    if (per > kAt) look(e);  // else the one batch is still at hand
#pragma unroll
    for (int q = 0; q < kAt; ++q) {
      const bool released = out >> q & 1u;
      if (!fits) {  // nothing is done: every row that keeps a page it was to drop is told
        if (page[q] >= 0) atomicOr(&a.status[(e + q) / a.max_blocks], SPEC_DEV_CAPACITY);
      } else if (page[q] >= 0) {
        if (released) a.pool[pos++] = page[q];
        *at[q] = -1;
      }
    }
  }
  if (fits && id == 0) *a.count = count + (int)total;
}

// ---------------------------------------------------------------------------
// Compact
// ---------------------------------------------------------------------------
struct CompactArgs {
  int32_t* table;
  int32_t *pool, *count, *page_map, *moved, *status;
  uint8_t* state;   // [num_blocks] kLive | kFree
  int* error;
  PageMove* moves;  // [num_blocks / 2]
  int* n_moves;
  long long entries;
  int num_blocks, bs, pool_cap;
};
constexpr int kLive = 1, kFree = 2;

__global__ void __launch_bounds__(kScanThreads) pages_compact_clear_kernel(const CompactArgs a) {
  let_next_launch();
  const int t = blockIdx.x * kScanThreads + threadIdx.x;
  for (int p = t; p < a.num_blocks; p += gridDim.x * kScanThreads) a.state[p] = 0;
  if (t == 0) *a.error = 0;
}

// Every page that a row names, then (second kernel) every page in the pool.
__global__ void __launch_bounds__(kScanThreads) pages_compact_live_kernel(const CompactArgs a) {
  let_next_launch();
  wait_for_last();
  const long long step = (long long)gridDim.x * kScanThreads;
  for (long long e = (long long)blockIdx.x * kScanThreads + threadIdx.x; e < a.entries; e += step) {
    const int p = a.table[e];
    if (p >= a.num_blocks) atomicOr(a.error, 1);
    else if (p >= 0) a.state[p] = kLive;
  }
}

// One cluster: the pool's pages, then the places.  S = live or free pages in
// increasing id; the first n of them (n = live pages) are the new places: the
// i-th free page among them receives the i-th live page beyond them.
__global__ void __launch_bounds__(kPlanThreads) pages_compact_plan_kernel(const CompactArgs a) {
  __shared__ ClusterScan scan;
  __shared__ int s_bad;
  let_next_launch();
  wait_for_last();
  cg::cluster_group cl = cg::this_cluster();
  const int G = (int)cl.num_blocks() * kPlanThreads, id = (int)cl.block_rank() * kPlanThreads + threadIdx.x;
  const int count = *(volatile int32_t*)a.count;
  int bad = *(volatile int*)a.error | (count < 0) | (count > a.pool_cap);
  // a page listed twice, or held and listed: nothing is done
  if (!bad) {
    for (int t = id; t < count; t += G) {
      const int p = a.pool[t];
      if (p < 0 || p >= a.num_blocks) {
        bad = 1;
        continue;
      }
      unsigned* word = reinterpret_cast<unsigned*>(a.state + (p & ~3));
      const unsigned old = atomicOr(word, (unsigned)kFree << (8 * (p & 3)));
      bad |= ((old >> (8 * (p & 3))) & 0xffu) != 0;
    }
  }
  __threadfence();
  if (threadIdx.x == 0) s_bad = 0;
  bad = __syncthreads_or(bad);
  cl.sync();
  if (bad && threadIdx.x < cl.num_blocks()) *cl.map_shared_rank(&s_bad, threadIdx.x) = 1;
  cl.sync();
  if (s_bad) {
    for (int p = id; p < a.num_blocks; p += G) a.page_map[p] = p;
    if (id == 0) {
      *a.status = SPEC_DEV_BAD_BLOCK;
      *a.moved = 0;
      *a.n_moves = 0;
    }
    return;
  }
  const int per = (a.num_blocks + G - 1) / G;
  const int p0 = (int)min((long long)a.num_blocks, (long long)id * per), p1 = min(a.num_blocks, p0 + per);
  auto state = [&](int p) -> int { return *(volatile uint8_t*)(a.state + p); };
  int live = 0, both = 0;
  for (int p = p0; p < p1; ++p) {
    const int s = state(p);
    live += s == kLive;
    both += s != 0;
  }
  long long n = 0, total = 0;
  cluster_scan(cl, scan, live, n);
  const long long place0 = cluster_scan(cl, scan, both, total);
  long long place = place0;
  int from = 0, to = 0;
  for (int p = p0; p < p1; ++p) {
    const int s = state(p);
    if (s == 0) continue;
    to += s == kFree && place < n;
    from += s == kLive && place >= n;
    ++place;
  }
  // destinations and sources are equally many
  long long m = 0, m2 = 0;
  long long at_from = cluster_scan(cl, scan, from, m);
  long long at_to = cluster_scan(cl, scan, to, m2);
  place = place0;
  for (int p = p0; p < p1; ++p) {
    const int s = state(p);
    if (s == kFree && place < n) a.moves[at_to++].dst = p;
    if (s == kLive && place >= n) {
      a.moves[at_from].src = p;
      a.moves[at_from++].rows = a.bs;
    } else {
      a.page_map[p] = p;
    }
    // the pages left over, highest id first: taking from the pool's end gives the lowest
    if (s != 0 && place >= n) a.pool[total - 1 - place] = p;
    place += s != 0;
  }
  __threadfence();
  cl.sync();
  for (long long i = id; i < m; i += G) a.page_map[__ldcg(&a.moves[i].src)] = __ldcg(&a.moves[i].dst);
  if (id == 0) {
    *a.status = 0;
    *a.moved = (int)m;
    *a.n_moves = (int)m;
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
struct Carve {  // 16-byte aligned pieces of the workspace
  char* base;
  size_t used = 0;
  template <typename T> T* take(size_t n) {
    T* p = reinterpret_cast<T*>(base + used);
    used += (n * sizeof(T) + 15) & ~(size_t)15;
    return p;
  }
};

static void carve_fork(ForkArgs& a, Carve& c) {
  a.n_moves = c.take<int>(1);
  a.mark = c.take<int>(a.B);
  a.need = c.take<long long>(a.N);
  a.moves = c.take<PageMove>(a.N);
}
static void carve_free(FreeArgs& a, Carve& c) {
  a.from = c.take<int>(a.B);
  a.entry = c.take<int>(a.B);
  a.mark = c.take<int>(a.B);
  a.first = c.take<int>(a.num_blocks);
}
static void carve_compact(CompactArgs& a, Carve& c) {
  a.n_moves = c.take<int>(1);
  a.error = c.take<int>(1);
  a.state = c.take<uint8_t>((size_t)a.num_blocks);
  a.moves = c.take<PageMove>((size_t)a.num_blocks / 2 + 1);
}

// Scalar checks shared by the three calls.
static spec_status pages_check(int B, int max_blocks, int block_size, int num_blocks, int N) {
  if (B < 0 || max_blocks <= 0 || num_blocks <= 0 || N < 0) return SPEC_ERR_INVALID_ARG;
  if (block_size < 8 || block_size > 65536 || (block_size & (block_size - 1))) return SPEC_ERR_UNSUPPORTED;
  // 32-bit counters step past the last entry by up to the threads of a grid
  if ((long long)B * max_blocks > (1LL << 30) || (long long)N * max_blocks > (1LL << 30) || num_blocks > (1 << 30))
    return SPEC_ERR_UNSUPPORTED;
  return SPEC_OK;
}
static spec_status caches_check(void* const* k, void* const* v, int layers, int Hkv, int D, spec_dtype dtype) {
  if (layers < 0 || Hkv <= 0) return SPEC_ERR_INVALID_ARG;
  if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return SPEC_ERR_UNSUPPORTED;
  if (Hkv > 65535 || layers > 32767) return SPEC_ERR_UNSUPPORTED;
  if (layers > 0 && (!k || !v)) return SPEC_ERR_INVALID_ARG;
  return SPEC_OK;
}

static bool sm_count(int* sms) {
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess &&
         cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess;
}

// A kernel of a call, in clusters of `cluster` CTAs; every one but the call's
// first is a programmatic dependent of the one before.
template <typename... P, typename... A>
static cudaError_t launch(void (*kern)(P...), int grid, int threads, int cluster, bool first, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = first ? 1 : 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, P(args)...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

static int scan_grid(long long n, int sms) {
  return (int)std::max(1LL, std::min<long long>(8LL * sms, (n + kScanThreads - 1) / kScanThreads));
}

}  // namespace spectree

using namespace spectree;

extern "C" {

size_t spec_pages_workspace_size(int B, int max_blocks, int num_blocks, int N) {
  (void)max_blocks;
  if (B < 0 || num_blocks < 0 || N < 0) return 256;
  ForkArgs f = {};
  FreeArgs r = {};
  CompactArgs c = {};
  f.B = r.B = B;
  f.N = N;
  r.num_blocks = c.num_blocks = num_blocks;
  Carve cf{nullptr}, cr{nullptr}, cc{nullptr};
  carve_fork(f, cf);
  carve_free(r, cr);
  carve_compact(c, cc);
  return std::max<size_t>(256, std::max(cf.used, std::max(cr.used, cc.used)));
}

spec_status spec_pages_fork(void* const* k_caches, void* const* v_caches, int layers, int32_t* block_table, int B,
                            int max_blocks, int block_size, int num_blocks, const int32_t* src, const int32_t* dst,
                            const int32_t* len, const int32_t* room, int N, int Hkv, int D, spec_dtype dtype,
                            int32_t* free_pool, int free_cap, int32_t* free_count, void* workspace,
                            size_t workspace_bytes, int32_t* status, void* stream) {
  SPEC_NVTX_RANGE("spec_pages_fork");
  spec_status sc = pages_check(B, max_blocks, block_size, num_blocks, N);
  if (sc == SPEC_OK) sc = caches_check(k_caches, v_caches, layers, Hkv, D, dtype);
  if (sc != SPEC_OK) return sc;
  if (free_cap < 0) return SPEC_ERR_INVALID_ARG;
  if (N == 0) return SPEC_OK;
  if (!block_table || !src || !dst || !len || !free_pool || !free_count || !status) return SPEC_ERR_INVALID_ARG;
  ForkArgs a = {};
  a.table = block_table;
  a.src = src;
  a.dst = dst;
  a.len = len;
  a.room = room;
  a.pool = free_pool;
  a.count = free_count;
  a.status = status;
  a.B = B;
  a.max_blocks = max_blocks;
  a.bs = block_size;
  a.num_blocks = num_blocks;
  a.N = N;
  a.pool_cap = free_cap;
  a.copies = layers > 0;
  Carve c{static_cast<char*>(workspace)};
  carve_fork(a, c);
  if (!workspace || workspace_bytes < c.used || (reinterpret_cast<uintptr_t>(workspace) & 15)) return SPEC_ERR_WORKSPACE;
  int sms = 0;
  if (!sm_count(&sms)) return SPEC_ERR_CUDA;
  cudaStream_t st = (cudaStream_t)stream;
  spec_workspace_canary(workspace, c.used, st);
  if (launch(pages_fork_kernel, kPlanCluster, kPlanThreads, kPlanCluster, true, st, a) != cudaSuccess) return SPEC_ERR_CUDA;
  if (layers > 0) {
    const int row_bytes = D * (dtype == SPEC_F32 ? 4 : 2);
    const long long head_bytes = (long long)block_size * row_bytes;
    const long long units = (long long)N * 2 * layers * Hkv * ((head_bytes + kMoveBytes - 1) / kMoveBytes);
    const int grid = (int)std::min<long long>((long long)kMoveCtas * sms, (units + 7) / 8);
    if (launch(page_move_kernel, grid, kMoveThreads, 1, false, st, (char* const*)k_caches, (char* const*)v_caches,
               2 * layers, a.moves, a.n_moves, Hkv, head_bytes, row_bytes, 0, nullptr, 0, nullptr, 0) != cudaSuccess)
      return SPEC_ERR_CUDA;
  }
  return SPEC_OK;
}

spec_status spec_pages_free(int32_t* block_table, int B, int max_blocks, int block_size, int num_blocks,
                            const int32_t* rows, const int32_t* keep_len, int N, int32_t* free_pool, int free_cap,
                            int32_t* free_count, void* workspace, size_t workspace_bytes, int32_t* status,
                            void* stream) {
  SPEC_NVTX_RANGE("spec_pages_free");
  const spec_status sc = pages_check(B, max_blocks, block_size, num_blocks, N);
  if (sc != SPEC_OK) return sc;
  if (free_cap < 0) return SPEC_ERR_INVALID_ARG;
  if (N == 0) return SPEC_OK;
  if (!block_table || !rows || !free_pool || !free_count || !status) return SPEC_ERR_INVALID_ARG;
  FreeArgs a = {};
  a.table = block_table;
  a.rows = rows;
  a.keep = keep_len;
  a.pool = free_pool;
  a.count = free_count;
  a.status = status;
  a.B = B;
  a.max_blocks = max_blocks;
  a.bs = block_size;
  a.num_blocks = num_blocks;
  a.N = N;
  a.pool_cap = free_cap;
  Carve c{static_cast<char*>(workspace)};
  carve_free(a, c);
  if (!workspace || workspace_bytes < c.used || (reinterpret_cast<uintptr_t>(workspace) & 15)) return SPEC_ERR_WORKSPACE;
  int sms = 0;
  if (!sm_count(&sms)) return SPEC_ERR_CUDA;
  cudaStream_t st = (cudaStream_t)stream;
  spec_workspace_canary(workspace, c.used, st);
  if (launch(pages_free_check_kernel, kPlanCluster, kPlanThreads, kPlanCluster, true, st, a) != cudaSuccess ||
      launch(pages_free_mark_kernel, scan_grid((long long)B * max_blocks, sms), kScanThreads, 1, false, st, a) != cudaSuccess ||
      launch(pages_free_release_kernel, kPlanCluster, kPlanThreads, kPlanCluster, false, st, a) != cudaSuccess)
    return SPEC_ERR_CUDA;
  return SPEC_OK;
}

spec_status spec_pages_compact(void* const* k_caches, void* const* v_caches, int layers, int32_t* block_table, int B,
                               int max_blocks, int block_size, int num_blocks, int Hkv, int D, spec_dtype dtype,
                               int32_t* free_pool, int free_cap, int32_t* free_count, int32_t* page_map,
                               int32_t* moved, void* workspace, size_t workspace_bytes, int32_t* status,
                               void* stream) {
  SPEC_NVTX_RANGE("spec_pages_compact");
  spec_status sc = pages_check(B, max_blocks, block_size, num_blocks, 0);
  if (sc == SPEC_OK) sc = caches_check(k_caches, v_caches, layers, Hkv, D, dtype);
  if (sc != SPEC_OK) return sc;
  if (free_cap < 0) return SPEC_ERR_INVALID_ARG;
  if ((B > 0 && !block_table) || !free_pool || !free_count || !page_map || !moved || !status)
    return SPEC_ERR_INVALID_ARG;
  CompactArgs a = {};
  a.table = block_table;
  a.pool = free_pool;
  a.count = free_count;
  a.page_map = page_map;
  a.moved = moved;
  a.status = status;
  a.entries = (long long)B * max_blocks;
  a.num_blocks = num_blocks;
  a.bs = block_size;
  a.pool_cap = free_cap;
  Carve c{static_cast<char*>(workspace)};
  carve_compact(a, c);
  if (!workspace || workspace_bytes < c.used || (reinterpret_cast<uintptr_t>(workspace) & 15)) return SPEC_ERR_WORKSPACE;
  int sms = 0;
  if (!sm_count(&sms)) return SPEC_ERR_CUDA;
  cudaStream_t st = (cudaStream_t)stream;
  spec_workspace_canary(workspace, c.used, st);
  if (launch(pages_compact_clear_kernel, scan_grid(num_blocks, sms), kScanThreads, 1, true, st, a) != cudaSuccess)
    return SPEC_ERR_CUDA;
  if (a.entries > 0 &&
      launch(pages_compact_live_kernel, scan_grid(a.entries, sms), kScanThreads, 1, false, st, a) != cudaSuccess)
    return SPEC_ERR_CUDA;
  const int row_bytes = D * (dtype == SPEC_F32 ? 4 : 2);
  if (launch(pages_compact_plan_kernel, kPlanCluster, kPlanThreads, kPlanCluster, false, st, a) != cudaSuccess ||
      launch(page_move_kernel, kMoveCtas * sms, kMoveThreads, 1, false, st, (char* const*)k_caches,
             (char* const*)v_caches, 2 * layers, a.moves, a.n_moves, Hkv, (long long)block_size * row_bytes, row_bytes,
             1, block_table, a.entries, page_map, num_blocks) != cudaSuccess)
    return SPEC_ERR_CUDA;
  return SPEC_OK;
}

}  // extern "C"
