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
#include <atomic>
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
enum Mode { kStats = 0, kSumsFew = 1, kSumsMany = 2, kHeld = 3 };
constexpr int kHeldRows = 32;        // rows whose scores are held, and the columns of a key tile's
constexpr int kHeldTiles = 512 / kHeldRows;  // key tiles of a CTA whose scores tensor memory holds

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
  int cluster;           // CTAs that hold one request's scores of a kv-head (0: none is held)
};

struct Request {
  int off, first, cnt, P, m;  // first counted token, counted tokens, prefix, tokens in all
  int quiet;                  // it came in flagged: nothing of it is written
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
  const bool held = prm.cluster > 0 && (R == 0 || (R <= kHeldRows && (total + BM - 1) / BM <= kHeldTiles * prm.cluster));
  if (MODE == kHeld) return held;
  if (held) return 0;
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
      // Every CTA has to number the items alike, so a status word, which a faster
      // CTA may set meanwhile, keeps a request's weights from being written but
      // does not take it out.
      const int came = *(const volatile int32_t*)&a.status[b];
      if (!bad && a.path)
        for (int i = r.m - r.cnt; i < r.m; ++i) bad |= weight_path_bad(a, r, i) ? SPEC_DEV_BAD_PATH : 0;
      if (bad && blockIdx.x == 0) atomicOr(&a.status[b], bad);
      q = {r.off, r.m - r.cnt, r.cnt, r.P, r.m, came};
      if (!bad) tiles = request_tiles<MODE>(prm, q);
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
  } else if (MODE == kSumsMany) {
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
  // Each kernel of a call but the first waits for the one before, whose results it
  // reads (the statistics need nothing of the held scores' kernel, and wait at
  // their end); each lets the next one launch as it starts.
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
        if (key < w.q.P + w.q.m && !w.q.quiet) a.weight[slot_at(w, key)] = sum;
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

  if (MODE == kStats) asm volatile("griddepcontrol.wait;" ::: "memory");
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

// ---------------------------------------------------------------------------
// Held scores: one pass over K.  A cluster of CTAs takes one request's kv-head
// (at most 32 rows), each CTA a run of its key tiles.  The scores of all tiles
// stay in tensor memory (32 columns a tile, up to 16 tiles); as a tile arrives,
// each thread adds 2^x of its key to the 32 row sums.  The CTAs exchange their
// sums (a value per row and CTA, by st.async to every CTA of the cluster), and
// the weights come from the scores still held: K is read once, nothing is read
// twice.  The ring of K tiles fills with the next request's while sums travel.
// ---------------------------------------------------------------------------
template <int D> struct HeldLayout {
  static constexpr int DH = D / 64;
  static constexpr int NST = D == 128 ? 5 : 8;
  static constexpr uint32_t kTile = BM * D * 2, kQ = kHeldRows * D * 2;
  static constexpr uint32_t kOffQ = NST * kTile;
  static constexpr uint32_t kBytes = kOffQ + 2 * kQ;
  static constexpr uint32_t kDyn = kBytes + 1024 < 120 * 1024 ? 120 * 1024 : kBytes + 1024;
  static_assert(kDyn + 16384 <= 227 * 1024, "dynamic and static shared memory within 227 KB");
};

// v[0] of lane e: the sum (or maximum) over the warp's lanes of what v[e] was.
template <bool MAX>
__device__ __forceinline__ float warp_columns(float (&v)[32], int lane) {
#pragma unroll
  for (int o = 16; o; o >>= 1)
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const bool up = lane & o;
      const float give = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
      const float got = __shfl_xor_sync(0xffffffffu, give, o);
      v[i] = MAX ? fmaxf(keep, got) : keep + got;
    }
  return v[0];
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// 4 bytes into CTA `rank`'s copy of a shared variable, completing on its copy of `bar`.
__device__ __forceinline__ void send_async(const float* var, uint64_t* bar, uint32_t rank, float value) {
  uint32_t to, on;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(smem_u32(var)), "r"(rank));
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(on) : "r"(smem_u32(bar)), "r"(rank));
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(to), "r"(__float_as_uint(value)), "r"(on)
               : "memory");
}
// mbar_wait for what other CTAs of the cluster wrote.
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  for (uint32_t i = 0; i < kWaitLimit; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    if (ok) return true;
    if ((i & 255u) == 255u && *abort_flag) return false;
  }
  *abort_flag = 1;
  return false;
}

constexpr int kHeldClusterMax = 16;

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    weight_held_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ Params prm) {
  using L = HeldLayout<D>;
  constexpr int NST = L::NST, N = kHeldRows, EW = 16;  // epilogue warps
  const WeightArgs& a = prm.a;
  extern __shared__ uint8_t dyn_raw[];
  __shared__ uint64_t full[NST], empty[NST], q_full[2], q_empty[2], s_full[kHeldTiles], s_empty[kHeldTiles], x_full[2], drain;
  __shared__ Table tab;
  __shared__ float s_red[EW][N], s_in[2][kHeldClusterMax][N];
  __shared__ __align__(16) float s_row[N];  // what the epilogue needs of each row: minus log2 of its sum, or its reference
  __shared__ int scan[kThreads / 32], abort_flag, issued[NST], s_redo;
  __shared__ uint32_t tmem_slot;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int C = prm.cluster, rank = (int)cluster_rank();
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn_raw) + 1023) & ~(uintptr_t)1023);
  const uint32_t sbase = smem_u32(smem);
  if (threadIdx.x == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
      issued[i] = -1;
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
      mbar_init(&x_full[i], 1);
    }
    for (int i = 0; i < kHeldTiles; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 4);
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
  cluster_sync_all();  // every CTA's barriers exist before another one's sums may arrive
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  auto wait = [&](uint64_t* bar, int phase) { return mbar_wait(bar, phase & 1, &abort_flag); };

  const int clusters = (int)gridDim.x / C, me = (int)blockIdx.x / C;
  auto dealt = [&](int round) { return round * clusters + (round & 1 ? clusters - 1 - me : me); };
  auto rounds_end = [&](int n) { return (n + clusters - 1) / clusters * clusters; };
  // this CTA's key tiles of an item: [t0, t0 + nt)
  auto share = [&](const Item& w, int& t0, int& nt) {
    const int tiles = (w.q.P + w.q.m + BM - 1) / BM, each = (tiles + C - 1) / C;
    t0 = rank * each;
    nt = max(0, min(each, tiles - t0));
  };

  int ld = 0;     // key tiles of this CTA so far (stream, MMA, epilogue)
  int units = 0;  // items with tiles here (Q, MMA); exchanges so far (epilogue)
  bool dead = false;
  for (int b0 = 0; b0 < a.B; b0 += kGroup) {
    const int n_items = build_table<kHeld>(prm, tab, b0, scan) * a.Hkv;
    if (warp == 0) {
      // ---------------------------------------------------------- K
      const int nb = BM / prm.box_rows;
      for (int round = 0, idx; (idx = dealt(round)) < rounds_end(n_items) && !dead; ++round) {
        if (idx >= n_items) continue;
        const Item w = find_item<kHeld>(prm, tab, b0, idx, lane);
        int t0, nt;
        share(w, t0, nt);
        if (w.q.cnt == 0 || nt == 0) continue;
        const int32_t* bt = a.block_table + (size_t)w.b * a.max_blocks;
        const int total = w.q.P + w.q.m, x0 = t0 * nb + lane, boxes = nt * nb;
        int bad = 0;
        auto page_of = [&](int x) -> int {
          const int k = x * prm.box_rows;
          if (k >= total) return -1;
          const int page = __ldg(bt + (k >> prm.bs_log2));
          if (page >= 0 && page < a.num_blocks) return page;
          bad = 1;
          return -1;
        };
        int pages = -1, ahead = lane < boxes ? page_of(x0) : -1;
        for (int j = 0; j < nt; ++j, ++ld) {
          const int st = ld % NST, at = j * nb & 31;
          if (at == 0) {
            pages = ahead;
            if (j * nb + 32 + lane < boxes) ahead = page_of(x0 + j * nb + 32);
          }
          bool go = true;
          if (lane == 0 && ld >= NST) go = wait(&empty[st], ld / NST - 1);
          dead = !__shfl_sync(0xffffffffu, (int)go, 0);
          if (dead) break;
          if (lane == 0) {
            issued[st] = ld;
            mbar_expect_tx(&full[st], L::kTile);
          }
          __syncwarp();
          const int page = __shfl_sync(0xffffffffu, pages, (at + lane) & 31);
          if (lane < nb) {
            const int k = (t0 + j) * BM + lane * prm.box_rows;
            const int y = page < 0 ? (int)prm.rows_total : ((page * a.Hkv + w.kvh) << prm.bs_log2) + (k & (a.block_size - 1));
#pragma unroll
            for (int h = 0; h < L::DH; ++h)
              tma_load_2d(sbase + st * L::kTile + h * (BM * 128) + lane * prm.box_rows * 128, &tmap_k, h * 64, y, &full[st]);
          }
        }
        if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(&a.status[w.b], SPEC_DEV_BAD_BLOCK);
      }
    } else if (warp == 2) {
      // ---------------------------------------------------------- Q: 32 rows, zeros behind the item's
      constexpr int CPR = D / 8, STEP = 32 / CPR;
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q);
      const int ch = lane % CPR;
      for (int round = 0, idx; (idx = dealt(round)) < rounds_end(n_items) && !dead; ++round) {
        if (idx >= n_items) continue;
        const Item w = find_item<kHeld>(prm, tab, b0, idx, lane);
        int t0, nt;
        share(w, t0, nt);
        if (w.q.cnt == 0 || nt == 0) continue;
        const int slot = units & 1, R = w.q.cnt * a.g;
        bool go = true;
        if (lane == 0 && units >= 2) go = wait(&q_empty[slot], (units >> 1) - 1);
        dead = !__shfl_sync(0xffffffffu, (int)go, 0);
        if (dead) break;
        const int32_t* path = a.path ? a.path + (size_t)w.b * a.path_stride + w.q.first : nullptr;
        const uint32_t dst = L::kOffQ + slot * L::kQ + (ch >> 3) * (N * 128);
#pragma unroll 4
        for (int i = lane / CPR; i < N; i += STEP) {
          const uint32_t at = dst + i * 128 + (((ch & 7) ^ (i & 7)) << 4);
          if (i < R) {
            const int tok = i / a.g, head = i % a.g;
            const size_t row = w.q.off + (path ? path[tok] : w.q.first + tok);
            cp_async16(sbase + at, q + (row * a.Hq + w.kvh * a.g + head) * D + ch * 8);
          } else {
            *reinterpret_cast<uint4*>(smem + at) = make_uint4(0, 0, 0, 0);
          }
        }
        cp_async_wait();
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[slot]);
        ++units;
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------- MMA: A = K tile, B = Q
      const uint64_t ring = smem_desc_sw128(sbase, 16, 1024), qd0 = smem_desc_sw128(sbase + L::kOffQ, 16, 1024);
      constexpr uint32_t idesc = idesc_bf16(N, 0);
      const bool leader = elect_one();
      for (int round = 0, idx; (idx = dealt(round)) < rounds_end(n_items); ++round) {
        if (idx >= n_items) continue;
        const Item w = find_item<kHeld>(prm, tab, b0, idx, lane);
        int t0, nt;
        share(w, t0, nt);
        if (w.q.cnt == 0 || nt == 0) continue;
        wait(&q_full[units & 1], units >> 1);
        const uint64_t qd = qd0 + (uint64_t)((units & 1) * (L::kQ >> 4));
        for (int j = 0; j < nt; ++j, ++ld) {
          const int st = ld % NST, s = ld % kHeldTiles;
          wait(&full[st], ld / NST);
          if (ld >= kHeldTiles) wait(&s_empty[s], ld / kHeldTiles - 1);
          tc_fence_after();
          if (leader) {
            const uint64_t kd = ring + (uint64_t)(st * (L::kTile >> 4));
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              umma_bf16(tmem + s * N, kd + (((kk >> 2) * (BM * 128) + (kk & 3) * 32) >> 4), qd + (((kk >> 2) * (N * 128) + (kk & 3) * 32) >> 4), idesc,
                        kk > 0 ? 1u : 0u);
            umma_commit(&s_full[s]);
            umma_commit(&empty[st]);
          }
          __syncwarp();
        }
        if (leader) umma_commit(&q_empty[units & 1]);
        __syncwarp();
        ++units;
      }
    } else if (warp >= 4) {
      // ---------------------------------------------------------- epilogue
      const int ew = warp - 4, wg = ew >> 2, quad = warp & 3, r = quad * 32 + lane;
      const uint32_t tS = tmem + ((uint32_t)(quad * 32) << 16);
      const float c2 = a.scale_log2;
      auto all_sync = [&]() { asm volatile("bar.sync 1, 512;" ::: "memory"); };
      // Row sums (or maxima) over the cluster, from each warp's own (row = lane):
      // warp 4 adds the CTA's, sends them to every CTA, and adds the CTAs'.  In
      // warp 4 the result of row `lane`, elsewhere nothing.
      auto exchange = [&](float v, bool max) -> float {
        s_red[ew][lane] = v;
        all_sync();
        if (ew != 0) return 0.0f;
#pragma unroll
        for (int k = 1; k < EW; ++k) v = max ? fmaxf(v, s_red[k][lane]) : v + s_red[k][lane];
        const int buf = units & 1;
        if (lane == 0) mbar_expect_tx(&x_full[buf], C * N * 4);
        __syncwarp();
        for (int k = 0; k < C; ++k) send_async(&s_in[buf][rank][lane], &x_full[buf], k, v);
        mbar_wait_cluster(&x_full[buf], (units >> 1) & 1, &abort_flag);
        float all = s_in[buf][0][lane];
        for (int k = 1; k < C; ++k) all = max ? fmaxf(all, s_in[buf][k][lane]) : all + s_in[buf][k][lane];
        __syncwarp();
        return all;
      };
      for (int round = 0, idx; (idx = dealt(round)) < rounds_end(n_items); ++round) {
        if (idx >= n_items) continue;
        const Item w = find_item<kHeld>(prm, tab, b0, idx, lane);
        int t0, nt;
        share(w, t0, nt);
        const int R = w.q.cnt * a.g, total = w.q.P + w.q.m;
        const size_t base = ((size_t)w.b * a.Hkv + w.kvh) * a.stride;
        auto old_weight = [&](int key) -> float { return a.before && key < w.q.P ? a.decay * a.before[base + key] : 0.0f; };
        if (w.q.cnt == 0) {  // no rows: the old weights alone
          for (int j = wg; j < nt; j += 4) {
            const int key = (t0 + j) * BM + r;
            if (key < total && !w.q.quiet) a.weight[base + key] = old_weight(key);
          }
          continue;
        }
        // the last slot that row `lane` sees
        const int lim = lane < R ? w.q.P + w.q.first + lane / a.g : -1;
        // f(e, scores of column e or -inf where the row does not see the key) over the
        // tiles of this warpgroup
        auto tile = [&](int j, float (&x)[N]) {  // tile j's scores, -inf where hidden
          uint32_t u[N];
          tmem_ld32(tS + (uint32_t)((ld + j) % kHeldTiles) * N, u);
          tmem_wait_ld(u);
          const int k0 = (t0 + j) * BM;
          if (k0 + BM - 1 > w.q.P + w.q.first) {
#pragma unroll
            for (int e = 0; e < N; ++e) {
              const int last = __shfl_sync(0xffffffffu, lim, e);
              x[e] = k0 + r <= last ? __uint_as_float(u[e]) : -INFINITY;
            }
          } else {
#pragma unroll
            for (int e = 0; e < N; ++e) x[e] = __uint_as_float(u[e]);
          }
        };
        float acc[N];
#pragma unroll
        for (int e = 0; e < N; ++e) acc[e] = 0.0f;
        for (int j = wg; j < nt; j += 4) {
          wait(&s_full[(ld + j) % kHeldTiles], (ld + j) / kHeldTiles);
          tc_fence_after();
          float x[N];
          tile(j, x);
#pragma unroll
          for (int e = 0; e < N; ++e) acc[e] += fast_exp2(x[e] * c2);
        }
        float old = wg < nt ? old_weight((t0 + wg) * BM + r) : 0.0f;
        float sum = exchange(warp_columns<false>(acc, lane), false);
        ++units;
        if (ew == 0) {
          const bool fits = lane >= R || (sum >= 1.0f / kSumTop && sum < kSumTop);
          s_row[lane] = lane < R ? -log2f(sum) : -INFINITY;
          const bool redo = !__all_sync(0xffffffffu, fits);
          if (lane == 0) s_redo = redo;
        }
        all_sync();
        if (s_redo) {  // a sum left fp32's middle: against the rows' maxima
#pragma unroll
          for (int e = 0; e < N; ++e) acc[e] = -INFINITY;
          for (int j = wg; j < nt; j += 4) {
            float x[N];
            tile(j, x);
#pragma unroll
            for (int e = 0; e < N; ++e) acc[e] = fmaxf(acc[e], x[e]);
          }
          float top = exchange(warp_columns<true>(acc, lane), true);
          ++units;
          top = lane < R && top > -INFINITY ? top * c2 : 0.0f;
          if (ew == 0) s_row[lane] = top;
          all_sync();
#pragma unroll
          for (int e = 0; e < N; ++e) acc[e] = 0.0f;
          for (int j = wg; j < nt; j += 4) {
            float x[N];
            tile(j, x);
#pragma unroll
            for (int e = 0; e < N; ++e) acc[e] += fast_exp2(fmaf(x[e], c2, -s_row[e]));
          }
          sum = exchange(warp_columns<false>(acc, lane), false);
          ++units;
          if (ew == 0) s_row[lane] = lane < R ? -(top + log2f(sum)) : -INFINITY;
          all_sync();
        }
        for (int j = wg; j < nt; j += 4) {
          const int key = (t0 + j) * BM + r;
          const float next = j + 4 < nt ? old_weight(key + 4 * BM) : 0.0f;
          float x[N];
          tile(j, x);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_empty[(ld + j) % kHeldTiles]);
          float2 p = make_float2(0.0f, 0.0f);
#pragma unroll
          for (int e = 0; e < N; e += 4) {
            const float4 n4 = *reinterpret_cast<const float4*>(&s_row[e]);
            p.x += fast_exp2(fmaf(x[e], c2, n4.x)) + fast_exp2(fmaf(x[e + 1], c2, n4.y));
            p.y += fast_exp2(fmaf(x[e + 2], c2, n4.z)) + fast_exp2(fmaf(x[e + 3], c2, n4.w));
          }
          if (key < total && !w.q.quiet) a.weight[base + key] = old + (p.x + p.y);
          old = next;
        }
        ld += nt;
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
    if (threadIdx.x == 0)
      for (int st = 0; st < NST; ++st)
        if (issued[st] >= 0) mbar_drain(&full[st], (issued[st] / NST) & 1);
    for (int b = threadIdx.x; b < a.B; b += kThreads) atomicOr(&a.status[b], SPEC_DEV_TIMEOUT);
  }
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
  __syncwarp();
  cluster_sync_all();  // no CTA's shared memory goes while another may still send to it
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
static void held_config(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr, int c) {
  cfg.gridDim = dim3(c, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = HeldLayout<D>::kDyn;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = c;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
}

// Clusters of c CTAs that device `dev` (the current one) runs at once; asked for
// once per device and size.
template <int D>
static int held_clusters(int dev, int c) {
  static std::atomic<int> known[64][kHeldClusterMax + 1];  // number + 1
  const bool keep = dev < 64;
  if (keep && known[dev][c] > 0) return known[dev][c] - 1;
  int n = 0;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  held_config<D>(cfg, attr, c);
  if (cudaFuncSetAttribute(weight_held_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)HeldLayout<D>::kDyn) != cudaSuccess ||
      cudaFuncSetAttribute(weight_held_kernel<D>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, weight_held_kernel<D>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  if (keep) known[dev][c] = n + 1;
  return n;
}

template <int D>
static cudaError_t launch_held(const CUtensorMap& mk, const Params& prm, int fit, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  held_config<D>(cfg, attr, prm.cluster);
  cfg.gridDim = dim3((unsigned)(std::min<long long>(fit, (long long)prm.a.B * prm.a.Hkv) * prm.cluster), 1, 1);
  cfg.stream = stream;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, weight_held_kernel<D>, mk, prm);
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
  const long long longest = (long long)a.max_prefix + a.n_max;
  // Scores are held where a request has few rows: by the fewest CTAs that can hold
  // the longest one's, and by more while the requests and heads alone leave SMs
  // idle.  A request with more rows or keys goes the other way, inside the kernels.
  bool first = true;
  if (a.g <= kHeldRows) {
    int c = 1;
    while (c < kHeldClusterMax && ((long long)c * kHeldTiles * BM < longest || 2LL * c * a.B * a.Hkv <= sms)) c *= 2;
    int fit = held_clusters<D>(dev, c);
    while (fit == 0 && c > 1) fit = held_clusters<D>(dev, c /= 2);
    if (fit == 0) return cudaErrorInvalidConfiguration;
    prm.cluster = c;
    e = launch_held<D>(mk, prm, fit, stream);
    if (e != cudaSuccess) return e;
    if (rows <= kHeldRows && longest <= (long long)c * kHeldTiles * BM) return cudaSuccess;  // every request's are held
    first = false;
  }
  const int dyn = (int)Layout<D>::kDyn;
  if (rows > 0) {
    const int tiles = (int)((rows + kJoinRows - 1) / kJoinRows);
    if ((long long)tiles * a.Hkv * a.B > INT32_MAX) return cudaErrorInvalidValue;
    e = launch(weight_tc_kernel<D, kStats>, sms, kThreads, dyn, first, stream, mk, mq, prm);
    if (e == cudaSuccess) e = launch(weight_join_kernel, (long long)tiles * a.Hkv * a.B, kJoinThreads, 0, false, stream, a, tiles);
  }
  if (e == cudaSuccess) e = launch(weight_tc_kernel<D, kSumsFew>, sms, kThreads, dyn, first && rows == 0, stream, mk, mq, prm);
  if (e == cudaSuccess && rows > 2 * BM) e = launch(weight_tc_kernel<D, kSumsMany>, sms, kThreads, dyn, false, stream, mk, mq, prm);
  return e;
}

}  // namespace wtc

cudaError_t launch_weight_tc(const WeightArgs& a, cudaStream_t stream) {
  return a.D == 64 ? wtc::launch_d<64>(a, stream) : wtc::launch_d<128>(a, stream);
}

}  // namespace spectree
