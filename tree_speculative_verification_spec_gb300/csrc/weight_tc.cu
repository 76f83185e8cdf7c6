// Attention weight of cached slots on the 5th-generation tensor cores (tcgen05),
// bf16 inputs, fp32 scores in tensor memory, never in global memory.
//
// Three forms of one kernel.  A CTA keeps up to two 128-row tiles in shared
// memory (resident) and walks a stream of 128-row tiles; each tcgen05.mma gives
// 128 x 128 scores, a thread of the epilogue owns one TMEM lane and reduces over
// its columns alone, so no reduction crosses lanes:
//   statistics      lanes = rows: resident Q (256 rows), stream K.  A row's
//                   reference and sum of 2^(x - reference).
//   sums, few rows  lanes = keys: resident Q (all rows, at most 256), stream K.
//                   A key's weight is done after its tile: sum over the columns
//                   (rows) of 2^(x - log2 of the row's sum).
//   sums, many      lanes = keys: resident K (256 keys), stream Q.  The weight
//                   stays in a register over every row tile that sees the keys.
// Four epilogue warpgroups, four score buffers.  Statistics and sums over many
// rows: each resident tile has two buffers in turn and two warpgroups, one for
// each half of the columns.  Sums over few rows: a warpgroup and a buffer take
// every fourth key tile.  (Two warpgroups, a whole buffer each, left the
// exponentials at 44 % and the tensor core at 44 % of a prompt's statistics: two
// warps a scheduler do not cover a score buffer's hand-over.)
//
// The reference of a row starts at 0 and is not a maximum: 2^(x - m) and its
// fp32 sum hold any m within 2^60 of the scores; a chunk whose sum leaves that
// range is done again against its own maximum, and the sum is scaled to it.
//
// Items (row tiles or key tiles of one request and kv-head) are numbered over
// the batch by a prefix sum that each CTA takes of its own, 256 requests at a
// time, and dealt out round-robin, the longest of a request first.
#include <algorithm>
#include <climits>

#include "tcgen05.cuh"
#include "weight.cuh"

namespace spectree {

namespace wtc {

using namespace tc5;

constexpr int BM = 128;
constexpr int kThreads = 640;        // warps: 0 stream, 1 MMA, 2 resident tiles, 3 sums of the rows, 4-19 epilogue (four warpgroups)
constexpr uint32_t kTmemCols = 512;  // four score buffers of 128 columns
constexpr int kLse = 4;              // row tiles whose sums are held for the epilogue
constexpr int kGroup = 256;          // requests numbered at a time
constexpr float kSumTop = 0x1p60f;
enum Mode { kStats = 0, kSumsFew = 1, kSumsMany = 2 };

template <int D> struct Layout {
  static constexpr int DH = D / 64;             // 128-byte halves of a row
  static constexpr int NST = D == 128 ? 4 : 6;  // stages of the stream
  static constexpr uint32_t kTile = BM * D * 2;
  static constexpr uint32_t kOffRing = 2 * kTile;
  static constexpr uint32_t kBytes = kOffRing + NST * kTile;
  static constexpr uint32_t kDyn = kBytes + 1024 < 120 * 1024 ? 120 * 1024 : kBytes + 1024;  // one CTA per SM (all of TMEM)
  static_assert(kDyn + 16384 <= 227 * 1024, "dynamic and static shared memory within 227 KB");
};

struct Params {
  WeightArgs a;
  long long rows_total;  // num_blocks * Hkv * block_size: rows of the 2-D cache view
  int box_rows;          // rows per TMA box: min(block_size, 128)
  int bs_log2;
  int q_tma;             // Q by TMA (packed rows, g divides 128), else by cp.async
  int key_chunk;         // keys per item of the sums over few rows
};

struct Request {
  int off, first, cnt, P, m;  // first counted token, counted tokens, prefix, tokens in all
};
struct Table {
  Request r[kGroup];
  int first[kGroup + 1];      // item tiles before each request
};

struct Item {
  Request q;
  int b, kvh, r0, k0, steps, split;
  int lo[2], hi[2];  // steps in which tile t has a job (statistics, sums over many rows)
  int rt;            // row tiles (sums over few rows)
};

// Tiles of request r in this form of the kernel.
template <int MODE>
__device__ __forceinline__ int request_tiles(const Params& prm, const Request& r) {
  const WeightArgs& a = prm.a;
  const int R = r.cnt * a.g, total = r.P + r.m;
  if (MODE == kStats) return (R + 2 * BM - 1) / (2 * BM);
  const bool few = R <= 2 * BM;
  if (MODE == kSumsFew) return few ? (total + prm.key_chunk - 1) / prm.key_chunk : 0;
  return few ? 0 : (total + 2 * BM - 1) / (2 * BM);
}

// Requests b0 .. of the group with their tiles, by every thread of the CTA.
// Returns the group's tiles.
template <int MODE>
__device__ __forceinline__ int build_table(const Params& prm, Table& tab, int b0, int* scan) {
  const WeightArgs& a = prm.a;
  const int c = threadIdx.x, b = b0 + c;
  int tiles = 0;
  if (c < kGroup) {
    Request q = {};
    if (b < a.B) {
      WeightRequest r;
      int bad = weight_check(a, b, r);
      const int came = *(const volatile int32_t*)&a.status[b];
      if (!bad && !came && a.path)
        for (int i = r.m - r.cnt; i < r.m; ++i) bad |= weight_path_bad(a, r, i) ? SPEC_DEV_BAD_PATH : 0;
      if (bad && blockIdx.x == 0) atomicOr(&a.status[b], bad);
      q = {r.off, r.m - r.cnt, r.cnt, r.P, r.m};
      if (!bad && !came) tiles = request_tiles<MODE>(prm, q);
    }
    tab.r[c] = q;
  }
  // inclusive scan over the group
  const int lane = c & 31, w = c >> 5;
  int incl = tiles;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) scan[w] = incl;
  __syncthreads();
  int before = 0;
  for (int k = 0; k < w; ++k) before += scan[k];
  if (c < kGroup) tab.first[c + 1] = before + incl;
  if (c == 0) tab.first[0] = 0;
  __syncthreads();
  return tab.first[kGroup];
}

// Item `idx` of the group (a whole warp).
template <int MODE>
__device__ __forceinline__ Item find_item(const Params& prm, const Table& tab, int b0, int idx, int lane) {
  const WeightArgs& a = prm.a;
  Item w = {};
  if (MODE == kStats) {
    w.split = idx % a.splits;
    idx /= a.splits;
  }
  w.kvh = idx % a.Hkv;
  const int tile = idx / a.Hkv;
  int cnt = 0;  // requests whose first tile is not above this one
#pragma unroll
  for (int r = lane; r < kGroup; r += 32) cnt += tab.first[r] <= tile;
  const int r = warp_sum_i(cnt) - 1;
  w.b = b0 + r;
  w.q = tab.r[r];
  const int at = tile - tab.first[r], R = w.q.cnt * a.g, total = w.q.P + w.q.m;
  if (MODE == kStats) {
    w.r0 = (tab.first[r + 1] - 1 - tile) * (2 * BM);  // the last rows see the most keys: first
    w.k0 = w.split * a.chunk;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int row = w.r0 + t * BM;
      if (row >= R) continue;
      const int end = min(w.q.P + w.q.first + (min(row + BM, R) - 1) / a.g + 1, w.k0 + a.chunk);
      if (end > w.k0) w.hi[t] = (end - w.k0 + BM - 1) / BM;
    }
    w.steps = max(w.hi[0], w.hi[1]);
  } else if (MODE == kSumsFew) {
    w.k0 = at * prm.key_chunk;
    w.steps = (min(prm.key_chunk, total - w.k0) + BM - 1) / BM;
    w.rt = (R + BM - 1) / BM;
  } else {
    w.k0 = at * (2 * BM);
    const int tok = max(0, w.k0 - w.q.P - w.q.first);  // the first counted token that sees the first key
    w.r0 = tok * a.g / BM * BM;
    w.steps = tok < w.q.cnt ? (R - w.r0 + BM - 1) / BM : 0;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int need = max(0, w.k0 + t * BM - w.q.P - w.q.first);
      if (w.k0 + t * BM < total && need < w.q.cnt) {
        w.lo[t] = (need * a.g - w.r0) / BM;
        w.hi[t] = w.steps;
      }
    }
  }
  return w;
}

template <int D, int MODE>
__global__ void __launch_bounds__(kThreads, 1)
    weight_tc_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_q,
                     const __grid_constant__ Params prm) {
  using L = Layout<D>;
  constexpr int NST = L::NST;
  const WeightArgs& a = prm.a;
  extern __shared__ uint8_t dyn_raw[];
  __shared__ uint64_t full[NST], empty[NST], res_full[2], res_empty[2], s_full[4], s_empty[4], drain;
  __shared__ Table tab;
  __shared__ uint64_t lse_full[kLse], lse_empty[kLse];
  __shared__ __align__(16) float s_lse[kLse][BM];  // minus log2 of the sums of a row tile's rows
  __shared__ __align__(16) int s_lim[kLse][BM];    // the last slot that each of them sees, -1: no row
  __shared__ float s_part[2][2][BM];
  __shared__ int scan[kThreads / 32], abort_flag, issued[NST], res_issued[2];
  __shared__ uint32_t tmem_slot;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn_raw) + 1023) & ~(uintptr_t)1023);
  const uint32_t sbase = smem_u32(smem);
  if (threadIdx.x == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
      issued[i] = -1;
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&res_full[i], 1);
      mbar_init(&res_empty[i], 1);
      res_issued[i] = -1;
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], MODE == kSumsFew ? 4 : 8);
    }
    for (int i = 0; i < kLse; ++i) {
      mbar_init(&lse_full[i], 1);
      mbar_init(&lse_empty[i], 16);
    }
    mbar_init(&drain, 1);
    abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  // Each kernel of a call but the first waits for the one before; each lets the
  // next one launch as it starts.
  if (MODE != kStats) asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // A wait that runs out sets the abort flag; every later wait then ends after a
  // few polls, and the items run to their ends on whatever they find (every
  // request is flagged, its weights are unspecified).
  auto wait = [&](uint64_t* bar, int phase) { return mbar_wait(bar, phase & 1, &abort_flag); };

  // Keys come by boxes of up to a page.  The page of an item's box x (boxes count
  // from slot 0 of the request), -1 behind its keys or at a bad id.
  const int nb = BM / prm.box_rows;
  auto box_page = [&](const Item& w, int x, int* bad) -> int {
    const int k = x * prm.box_rows;
    if (k >= w.q.P + w.q.m) return -1;
    const int page = __ldg(a.block_table + (size_t)w.b * a.max_blocks + (k >> prm.bs_log2));
    if (page >= 0 && page < a.num_blocks) return page;
    *bad = 1;
    return -1;
  };
  // Key tile j of an item: lane i < nb copies box i from its page; without one it
  // reads behind the cache (zeros).
  auto load_keys = [&](const Item& w, int j, int page, uint32_t dst, uint64_t* bar) {
    if (lane < nb) {
      const int k = w.k0 + j * BM + lane * prm.box_rows;
      const int y = page < 0 ? (int)prm.rows_total : ((page * a.Hkv + w.kvh) << prm.bs_log2) + (k & (a.block_size - 1));
#pragma unroll
      for (int h = 0; h < L::DH; ++h) tma_load_2d(dst + h * (BM * 128) + lane * prm.box_rows * 128, &tmap_k, h * 64, y, bar);
    }
  };
  // Rows r .. r + 127 of an item (row = (counted token, head of the group)); rows
  // behind its last are whatever lies there.  True: `bar` still has to
  // be arrived on.
  auto load_rows = [&](const Item& w, int r, uint32_t dst, uint64_t* bar) -> bool {
    if (prm.q_tma) {
      if (lane == 0)
#pragma unroll
        for (int h = 0; h < L::DH; ++h)
          tma_load_3d(dst + h * (BM * 128), &tmap_q, h * 64, w.kvh * a.g, w.q.off + w.q.first + r / a.g, bar);
      return false;
    }
    constexpr int CPR = D / 8;      // 16-byte chunks per row
    constexpr int STEP = 32 / CPR;  // rows per round
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q);
    const int ch = lane % CPR, R = w.q.cnt * a.g;
    const int32_t* path = a.path ? a.path + (size_t)w.b * a.path_stride + w.q.first : nullptr;
#pragma unroll 4
    for (int i = lane / CPR; i < min(BM, R - r); i += STEP) {
      const uint32_t at = dst + (ch >> 3) * (BM * 128) + i * 128 + (((ch & 7) ^ (i & 7)) << 4);
      const int tok = (r + i) / a.g, head = (r + i) % a.g;
      const size_t row = w.q.off + (path ? path[tok] : w.q.first + tok);
      cp_async16(at, q + (row * a.Hq + w.kvh * a.g + head) * D + ch * 8);
    }
    return true;
  };
  auto copies_done = [&](uint64_t* bar) {
    cp_async_wait();
    fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };

  auto resident = [&](const Item& w) { return MODE == kSumsFew ? w.rt : w.hi[1] > 0 ? 2 : 1; };  // tiles
  // Round k deals items k grid .. (k + 1) grid - 1 to the CTAs, every other round
  // backwards: costs fall along a request, so a CTA's sums come out alike.
  const int grid = (int)gridDim.x, me = (int)blockIdx.x;
  auto dealt = [&](int round) { return round * grid + (round & 1 ? grid - 1 - me : me); };
  auto rounds_end = [&](int n) { return (n + grid - 1) / grid * grid; };

  int rs = 0;                           // resident tiles so far: tile i of an item lies in slot (rs + i) & 1
  int ld = 0;                           // stream tiles so far
  int jobs[4] = {0, 0, 0, 0};           // score tiles so far: of each resident tile, or of each buffer (MMA warp)
  int c = 0;                            // the same of this warpgroup's (epilogue)
  int lt = 0;                           // row tiles of sums so far
  bool dead = false;                    // a producer that gave up
  for (int b0 = 0; b0 < a.B; b0 += kGroup) {
    const int tiles = build_table<MODE>(prm, tab, b0, scan);
    const int n_items = tiles * a.Hkv * (MODE == kStats ? a.splits : 1);
    if (warp == 0) {
      // ---------------------------------------------------------- stream
      for (int round = 0, idx; (idx = dealt(round)) < rounds_end(n_items) && !dead; ++round) {
        if (idx >= n_items) continue;
        const Item w = find_item<MODE>(prm, tab, b0, idx, lane);
        if (MODE == kSumsFew && w.rt == 0) continue;
        // the pages of 32 boxes at a time, one to a lane, and the next 32 ahead
        int bad = 0, pages = -1, ahead = -1;
        const int x0 = w.k0 / prm.box_rows + lane, boxes = w.steps * nb;
        if (MODE != kSumsMany && lane < boxes) ahead = box_page(w, x0, &bad);
        for (int j = 0; j < w.steps; ++j, ++ld) {
          const int st = ld % NST, at = j * nb & 31;
          if (MODE != kSumsMany && at == 0) {
            pages = ahead;
            if (j * nb + 32 + lane < boxes) ahead = box_page(w, x0 + j * nb + 32, &bad);
          }
          bool go = true;
          if (lane == 0 && ld >= NST) go = wait(&empty[st], ld / NST - 1);
          dead = !__shfl_sync(0xffffffffu, (int)go, 0);
          if (dead) break;
          const uint32_t dst = sbase + L::kOffRing + st * L::kTile;
          if (lane == 0) issued[st] = ld;
          if (MODE == kSumsMany) {
            if (lane == 0 && prm.q_tma) mbar_expect_tx(&full[st], L::kTile);
            __syncwarp();
            if (load_rows(w, w.r0 + j * BM, dst, &full[st])) copies_done(&full[st]);
          } else {
            if (lane == 0) mbar_expect_tx(&full[st], L::kTile);
            __syncwarp();
            load_keys(w, j, __shfl_sync(0xffffffffu, pages, (at + lane) & 31), dst, &full[st]);
          }
        }
        if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(&a.status[w.b], SPEC_DEV_BAD_BLOCK);
      }
    } else if (warp == 2) {
      // ---------------------------------------------------------- resident tiles
      for (int round = 0, idx; (idx = dealt(round)) < rounds_end(n_items) && !dead; ++round) {
        if (idx >= n_items) continue;
        const Item w = find_item<MODE>(prm, tab, b0, idx, lane);
        if (w.steps == 0 || (MODE == kSumsFew && w.rt == 0)) continue;
        const int n = resident(w);
        int bad = 0;
        for (int t = 0; t < n; ++t, ++rs) {
          const int slot = rs & 1;
          bool go = true;
          if (lane == 0 && rs >= 2) go = wait(&res_empty[slot], (rs >> 1) - 1);
          dead = !__shfl_sync(0xffffffffu, (int)go, 0);
          if (dead) break;
          if (lane == 0) res_issued[slot] = rs >> 1;
          if (lane == 0 && (MODE == kSumsMany || prm.q_tma)) mbar_expect_tx(&res_full[slot], L::kTile);
          __syncwarp();
          if (MODE == kSumsMany) {
            const int x = w.k0 / prm.box_rows + t * nb + lane;
            load_keys(w, t, lane < nb ? box_page(w, x, &bad) : -1, sbase + slot * L::kTile, &res_full[slot]);
          } else if (load_rows(w, w.r0 + t * BM, sbase + slot * L::kTile, &res_full[slot])) {
            copies_done(&res_full[slot]);
          }
        }
        if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(&a.status[w.b], SPEC_DEV_BAD_BLOCK);
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------- MMA
      const uint64_t res = smem_desc_sw128(sbase, 16, 1024), ring = smem_desc_sw128(sbase + L::kOffRing, 16, 1024);
      const bool leader = elect_one();
      for (int round = 0, idx; (idx = dealt(round)) < rounds_end(n_items); ++round) {
        if (idx >= n_items) continue;
        const Item w = find_item<MODE>(prm, tab, b0, idx, lane);
        if (w.steps == 0 || (MODE == kSumsFew && w.rt == 0)) continue;
        const int R = w.q.cnt * a.g, n = resident(w);
        for (int t = 0; t < n; ++t) wait(&res_full[(rs + t) & 1], (rs + t) >> 1);
        for (int j = 0; j < w.steps; ++j, ++ld) {
          const int st = ld % NST;
          wait(&full[st], ld / NST);
          const uint64_t sd = ring + (uint64_t)(st * (L::kTile >> 4));
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (MODE == kSumsFew ? t >= w.rt : j < w.lo[t] || j >= w.hi[t]) continue;
            // buffer, and the number of its jobs before this one
            int buf, before;
            if (MODE == kSumsFew) {
              buf = w.rt == 2 ? (j & 1) * 2 + t : j & 3;
              before = buf == 0 ? jobs[0]++ : buf == 1 ? jobs[1]++ : buf == 2 ? jobs[2]++ : jobs[3]++;
            } else {
              const int c = jobs[t]++;
              buf = t * 2 + (c & 1);
              before = c >> 1;
            }
            if (before > 0) wait(&s_empty[buf], before - 1);
            tc_fence_after();
            const uint64_t rd = res + (uint64_t)(((rs + t) & 1) * (L::kTile >> 4));
            const uint32_t d = tmem + buf * BM;
            // few rows: only the columns that hold some, 32 at a time
            const uint32_t n = MODE == kSumsFew ? min(BM, (R - t * BM + 31) / 32 * 32) : BM;
            const uint32_t idesc = idesc_bf16(BM, 0) & ~(0x3fu << 17) | (n >> 3) << 17;
            if (leader) {
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t o = ((kk >> 2) * (BM * 128) + (kk & 3) * 32) >> 4;
                umma_bf16(d, (MODE == kSumsFew ? sd : rd) + o, (MODE == kSumsFew ? rd : sd) + o, idesc, kk > 0 ? 1u : 0u);
              }
              umma_commit(&s_full[buf]);
            }
            __syncwarp();
          }
          if (leader) umma_commit(&empty[st]);
          __syncwarp();
        }
        for (int t = 0; t < n; ++t, ++rs)
          if (leader) umma_commit(&res_empty[rs & 1]);
        __syncwarp();
      }
    } else if (warp == 3 && MODE != kStats) {
      // ---------------------------------------------------------- sums of the rows
      for (int round = 0, idx; (idx = dealt(round)) < rounds_end(n_items) && !dead; ++round) {
        if (idx >= n_items) continue;
        const Item w = find_item<MODE>(prm, tab, b0, idx, lane);
        const int n = MODE == kSumsFew ? w.rt : w.steps, R = w.q.cnt * a.g;
        for (int t = 0; t < n; ++t, ++lt) {
          const int at = lt % kLse;
          float nl[BM / 32];
          int lim[BM / 32];
          const int row0 = w.r0 + t * BM + lane;
          const float* lse = a.ws_lse + weight_ws_row(a, w.kvh, w.q.off, w.q.first) + row0;
#pragma unroll
          for (int e = 0; e < BM / 32; ++e) {
            const bool there = row0 + e * 32 < R;
            lim[e] = there ? w.q.P + w.q.first + (row0 + e * 32) / a.g : -1;
            nl[e] = there ? lse[e * 32] : -INFINITY;
          }
          bool go = true;
          if (lane == 0 && lt >= kLse) go = wait(&lse_empty[at], lt / kLse - 1);
          dead = !__shfl_sync(0xffffffffu, (int)go, 0);
          if (dead) break;
#pragma unroll
          for (int e = 0; e < BM / 32; ++e) {
            s_lse[at][e * 32 + lane] = nl[e];
            s_lim[at][e * 32 + lane] = lim[e];
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&lse_full[at]);
        }
      }
    } else if (warp >= 4) {
      // ---------------------------------------------------------- epilogue
      const int wg = (warp - 4) >> 2, quad = warp & 3, r = quad * 32 + lane;  // warpgroup, TMEM lane
      const int g = wg & 1, half = wg >> 1;  // resident tile and half of its columns
      const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
      const float c2 = a.scale_log2;
      const float2 c22 = make_float2(c2, c2);
      // the next score buffer of this warpgroup: its TMEM columns, and its return
      auto take = [&]() -> uint32_t {
        const int buf = MODE == kSumsFew ? wg : g * 2 + (c & 1);
        wait(&s_full[buf], MODE == kSumsFew ? c : c >> 1);
        tc_fence_after();
        return tmem + buf * BM + lane_off;
      };
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_empty[MODE == kSumsFew ? wg : g * 2 + (c & 1)]);
        ++c;
      };
      auto lse_done = [&](int i) {  // this warp has read row tile i's sums
        __syncwarp();
        if (lane == 0) mbar_arrive(&lse_empty[i % kLse]);
      };
      // sum over 32 columns of 2^(x c + nl), the columns that see `key` alone where
      // `masked`
      auto column_sum = [&](const uint32_t (&x)[32], const float* nl, const int* lim, bool masked, int key, float2& acc) {
        if (masked) {
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float p0 = fast_exp2(fmaf(__uint_as_float(x[e]), c2, nl[e])), p1 = fast_exp2(fmaf(__uint_as_float(x[e + 1]), c2, nl[e + 1]));
            acc.x += key <= lim[e] ? p0 : 0.0f;
            acc.y += key <= lim[e + 1] ? p1 : 0.0f;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 n4 = *reinterpret_cast<const float4*>(nl + e);
            const float2 z0 = __ffma2_rn(make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), c22, make_float2(n4.x, n4.y));
            const float2 z1 = __ffma2_rn(make_float2(__uint_as_float(x[e + 2]), __uint_as_float(x[e + 3])), c22, make_float2(n4.z, n4.w));
            acc = __fadd2_rn(acc, make_float2(fast_exp2(z0.x), fast_exp2(z0.y)));
            acc = __fadd2_rn(acc, make_float2(fast_exp2(z1.x), fast_exp2(z1.y)));
          }
        }
      };
      auto slot_at = [&](const Item& w, int key) { return ((size_t)w.b * a.Hkv + w.kvh) * a.stride + key; };
      auto old_weight = [&](const Item& w, int key) -> float {
        return a.before && key < w.q.P ? a.decay * a.before[slot_at(w, key)] : 0.0f;
      };
      auto put = [&](const Item& w, int key, float sum) {
        if (key < w.q.P + w.q.m) a.weight[slot_at(w, key)] = sum;
      };

      for (int round = 0, idx; (idx = dealt(round)) < rounds_end(n_items); ++round) {
        if (idx >= n_items) continue;
        const Item w = find_item<MODE>(prm, tab, b0, idx, lane);
        const int R = w.q.cnt * a.g, lo = g ? w.lo[1] : w.lo[0], hi = g ? w.hi[1] : w.hi[0];
        if (MODE == kStats) {
          if (hi == 0) continue;
          const int row = w.r0 + g * BM + r;
          const bool valid = row < R;
          const int tok = w.q.first + (valid ? row / a.g : w.q.cnt - 1);
          const int lim = w.q.P + tok + 1 - w.k0;  // visible keys of this range
          float m = 0.0f, l = 0.0f;
          auto weights = [&](uint32_t (&x)[32], int vis) -> float {
            if (!__all_sync(0xffffffffu, vis >= 32)) {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (e >= vis) x[e] = 0xff800000u;
            }
            const float2 neg = make_float2(-m, -m);
            float2 a0 = make_float2(0.0f, 0.0f), a1 = a0;
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const float2 z0 = __ffma2_rn(make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), c22, neg);
              const float2 z1 = __ffma2_rn(make_float2(__uint_as_float(x[e + 2]), __uint_as_float(x[e + 3])), c22, neg);
              a0 = __fadd2_rn(a0, make_float2(fast_exp2(z0.x), fast_exp2(z0.y)));
              a1 = __fadd2_rn(a1, make_float2(fast_exp2(z1.x), fast_exp2(z1.y)));
            }
            return (a0.x + a0.y) + (a1.x + a1.y);
          };
          auto chunk = [&](uint32_t (&x)[32], int vis) {
            float sum = weights(x, vis);
            const bool unfit = valid && (sum >= kSumTop || (l == 0.0f && vis > 0 && sum < 1.0f / kSumTop));
            if (__any_sync(0xffffffffu, unfit)) {  // against the chunk's maximum
              float mx = -INFINITY;
#pragma unroll
              for (int e = 0; e < 32; ++e) mx = fmaxf(mx, __uint_as_float(x[e]));  // hidden ones are -inf
              mx *= c2;
              if (l == 0.0f) {
                if (mx > -INFINITY) m = mx;
              } else if (mx > m) {
                l *= fast_exp2(m - mx);
                m = mx;
              }
              sum = weights(x, vis);
            }
            l += sum;
          };
          const bool idle = !__any_sync(0xffffffffu, valid);  // a warp without rows only passes the buffers on
          for (int j = 0; j < hi; ++j) {
            const uint32_t t0 = take() + half * 64;
            if (!idle) {
              const int vis = lim - j * BM - half * 64;
              uint32_t x[32];
#pragma unroll 1
              for (int e = 0; e < 64; e += 32) {
                tmem_ld32(t0 + e, x);
                tmem_wait_ld(x);
                chunk(x, vis - e);
              }
            }
            release();
          }
          if (valid)
            a.ws_ml[((size_t)w.split * a.T * a.Hq + weight_ws_row(a, w.kvh, w.q.off, w.q.first) + row) * 2 + half] = make_float2(m, l);
        } else if (MODE == kSumsFew) {
          if (w.rt == 0) {  // no rows: the old weights alone
            for (int j = wg; j < w.steps; j += 4) put(w, w.k0 + j * BM + r, old_weight(w, w.k0 + j * BM + r));
            continue;
          }
          // one row tile: every fourth key tile; two: one of them for every other
          const bool two = w.rt == 2;
          const int j0 = two ? wg >> 1 : wg, dj = two ? 2 : 4, t = two ? wg & 1 : 0, at = (lt + t) % kLse;
          float old = t == 0 ? old_weight(w, w.k0 + j0 * BM + r) : 0.0f;
          wait(&lse_full[at], (lt + t) / kLse);
          const int cols = min(BM, R - t * BM);
          for (int j = j0; j < w.steps; j += dj) {
            const int k0 = w.k0 + j * BM, key = k0 + r;
            const float next = t == 0 && j + dj < w.steps ? old_weight(w, key + dj * BM) : 0.0f;
            float2 acc = make_float2(0.0f, 0.0f);
            const uint32_t t0 = take();
            // rows that do not see the tile's last key, or columns without a row
            const bool masked = k0 + BM - 1 > w.q.P + w.q.first || (cols & 31) != 0;
#pragma unroll 1
            for (int e = 0; e < cols; e += 32) {
              uint32_t x[32];
              tmem_ld32(t0 + e, x);
              tmem_wait_ld(x);
              column_sum(x, &s_lse[at][e], &s_lim[at][e], masked, key, acc);
            }
            release();
            float sum = acc.x + acc.y;
            if (two) {  // the other row tile's share; the buffer is read before the barrier of the pair's next tile
              float* part = s_part[wg >> 1][(j >> 1) & 1];
              if (t == 1) part[r] = sum;
              asm volatile("bar.sync %0, 256;" ::"r"(1 + (wg >> 1)) : "memory");
              if (t == 0) sum += part[r];
            }
            if (t == 0) put(w, key, old + sum);
            old = next;
          }
          // both row tiles' sums go back, read here or not
          if (two) wait(&lse_full[(lt + 1 - t) % kLse], (lt + 1 - t) / kLse);
          for (int t = 0; t < w.rt; ++t, ++lt) lse_done(lt);
        } else {
          const int k0 = w.k0 + g * BM, key = k0 + r;
          const float old = half == 0 ? old_weight(w, key) : 0.0f;
          float2 acc = make_float2(0.0f, 0.0f);
          for (int j = 0; j < w.steps; ++j, ++lt) {
            const int at = lt % kLse;
            wait(&lse_full[at], lt / kLse);
            if (j >= lo && j < hi) {
              const int row0 = w.r0 + j * BM;
              const uint32_t t0 = take();
              const bool masked = k0 + BM - 1 > w.q.P + w.q.first + row0 / a.g || row0 + BM > R;
#pragma unroll 1
              for (int e = half * 64; e < half * 64 + 64; e += 32) {
                uint32_t x[32];
                tmem_ld32(t0 + e, x);
                tmem_wait_ld(x);
                column_sum(x, &s_lse[at][e], &s_lim[at][e], masked, key, acc);
              }
              release();
            }
            lse_done(lt);
          }
          // the two halves of the columns, through shared memory
          if (half == 1) s_part[g][0][r] = acc.x + acc.y;
          asm volatile("bar.sync %0, 256;" ::"r"(1 + g) : "memory");
          if (half == 0) put(w, key, old + (acc.x + acc.y) + s_part[g][0][r]);
          asm volatile("bar.sync %0, 256;" ::"r"(1 + g) : "memory");
        }
      }
    }
    __syncthreads();  // the table has been read
  }

  if (warp == 1 && elect_one()) {  // every MMA has completed before TMEM is freed
    umma_commit(&drain);
    mbar_drain(&drain, 0);
  }
  tc_fence_before();
  __syncthreads();
  if (abort_flag) {
    if (threadIdx.x == 0) {  // copies in flight land before the CTA exits
      for (int st = 0; st < NST; ++st)
        if (issued[st] >= 0) mbar_drain(&full[st], (issued[st] / NST) & 1);
      for (int i = 0; i < 2; ++i)
        if (res_issued[i] >= 0) mbar_drain(&res_full[i], res_issued[i] & 1);
    }
    for (int b = threadIdx.x; b < a.B; b += kThreads) atomicOr(&a.status[b], SPEC_DEV_TIMEOUT);
  }
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

// Minus log2 of every counted row's sum, from the parts that the splits with some
// of its keys left: 8 lanes a row, 32 rows a CTA.
constexpr int kJoinThreads = 256, kJoinRows = kJoinThreads / 8;
__global__ void __launch_bounds__(kJoinThreads) weight_join_kernel(const WeightArgs a, int tiles) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tile = blockIdx.x % tiles, kvh = blockIdx.x / tiles % a.Hkv, b = blockIdx.x / tiles / a.Hkv;
  WeightRequest r;
  const bool bad = weight_check(a, b, r) != 0;
  const int row = tile * kJoinRows + threadIdx.x / 8, part = threadIdx.x % 8;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (bad || tile * kJoinRows >= r.cnt * a.g) return;
  const bool there = row < r.cnt * a.g;
  const int first = r.m - r.cnt;
  const int splits = there ? min(a.splits, (r.P + first + row / a.g) / a.chunk + 1) : 0;
  const size_t at = weight_ws_row(a, kvh, r.off, first) + row, step = (size_t)a.T * a.Hq;
  const float4* ml = reinterpret_cast<const float4*>(a.ws_ml) + at;
  float2 x = make_float2(0.0f, 0.0f);
#pragma unroll 4
  for (int s = part; s < splits; s += 8) {
    const float4 y = ml[s * step];
    x = weight_join(x, weight_join(make_float2(y.x, y.y), make_float2(y.z, y.w)));
  }
#pragma unroll
  for (int o = 4; o; o >>= 1) {
    const float2 y = make_float2(__shfl_xor_sync(0xffffffffu, x.x, o), __shfl_xor_sync(0xffffffffu, x.y, o));
    x = weight_join(x, y);
  }
  if (there && part == 0) a.ws_lse[at] = -(x.x + log2f(x.y));
}

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeFn encode_fn() {
  static const EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

static bool make_map(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                     const cuuint32_t* box) {
  const EncodeFn enc = encode_fn();
  const cuuint32_t one[3] = {1, 1, 1};
  return enc && enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box, one,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A kernel of a call; every one but the first is a programmatic dependent of the
// one before.
template <typename... P, typename... A>
static cudaError_t launch(void (*kern)(P...), long long grid, int threads, int dyn, bool first, cudaStream_t stream, const A&... args) {
  if (dyn > 0) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, dyn);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = dyn;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = first ? 0 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int D>
static cudaError_t launch_d(const WeightArgs& a, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  Params prm = {};
  prm.a = a;
  prm.box_rows = std::min(a.block_size, BM);
  while ((1 << prm.bs_log2) < a.block_size) ++prm.bs_log2;
  prm.rows_total = (long long)a.num_blocks * a.Hkv * a.block_size;
  prm.q_tma = !a.path && BM % a.g == 0 && a.T > 0;
  // sums over few rows: some four items for every CTA, of 256 to 2048 keys
  const long long keys = ((long long)a.max_prefix + a.n_max) * a.B * a.Hkv / (4LL * sms);
  prm.key_chunk = (int)std::min(2048LL, std::max(256LL, (keys + 255) / 256 * 256));
  alignas(64) CUtensorMap mk, mq;
  {
    const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)prm.rows_total}, strides[1] = {(cuuint64_t)D * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)prm.box_rows};
    if (!make_map(&mk, a.k_cache, 2, dims, strides, box)) return cudaErrorInvalidValue;
  }
  if (prm.q_tma) {  // Q [T][Hq][D] as (columns, heads, tokens)
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)a.Hq, (cuuint64_t)a.T};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)a.Hq * D * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)a.g, (cuuint32_t)(BM / a.g)};
    if (!make_map(&mq, a.q, 3, dims, strides, box)) return cudaErrorInvalidValue;
  } else {
    mq = mk;  // not read
  }
  const long long rows = (long long)(a.window > 0 ? std::min(a.window, a.n_max) : a.n_max) * a.g;  // the most that a request has
  const int dyn = (int)Layout<D>::kDyn;
  if (rows > 0) {
    const int tiles = (int)((rows + kJoinRows - 1) / kJoinRows);
    if ((long long)tiles * a.Hkv * a.B > INT32_MAX) return cudaErrorInvalidValue;
    e = launch(weight_tc_kernel<D, kStats>, sms, kThreads, dyn, true, stream, mk, mq, prm);
    if (e == cudaSuccess) e = launch(weight_join_kernel, (long long)tiles * a.Hkv * a.B, kJoinThreads, 0, false, stream, a, tiles);
  }
  if (e == cudaSuccess) e = launch(weight_tc_kernel<D, kSumsFew>, sms, kThreads, dyn, rows == 0, stream, mk, mq, prm);
  if (e == cudaSuccess && rows > 2 * BM) e = launch(weight_tc_kernel<D, kSumsMany>, sms, kThreads, dyn, false, stream, mk, mq, prm);
  return e;
}

}  // namespace wtc

cudaError_t launch_weight_tc(const WeightArgs& a, cudaStream_t stream) {
  return a.D == 64 ? wtc::launch_d<64>(a, stream) : wtc::launch_d<128>(a, stream);
}

}  // namespace spectree
