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
// time, and dealt out back and forth, the longest of a request first.
//
// Requests of at most 32 rows (single tokens, accepted paths) have a kernel of
// their own, which reads K once: see "Held scores" below.
//
// What bounds them, and what they measured (32/8 heads, D 128, one GB300):
//   every row of a prompt of 8192: statistics 229 us, sums 273 (241 and 298 with
//   one MMA warp for both tiles).  No pipe is full (tensor core and exponentials
//   some 50 %, issue slots 60 %): the chain of a score buffer from hand to hand.
//   Sums have 256 items for 152 CTAs, the first keys' the longest (15 %; items of
//   128 keys end more evenly but stream Q twice: 380 us against 311 at that step).
//   the last 32 rows of four prompts of 8704 slots, 64/8 heads: 29 us, 37 us, and
//   the join of the row sums between them.
//   Two passes over K against 512 rows' of 8000 keys: 185 and 199 us, 5.8 TB/s.
#include <algorithm>
#include <atomic>
#include <climits>

#include "tcgen05.cuh"
#include "weight.cuh"

namespace spectree {

namespace wtc {

using namespace tc5;

constexpr int BM = 128;
constexpr int kThreads = 640;        // warps: 0 stream, 1 MMA, 2 resident tiles (and sums of the rows), 3 MMA of the second tile (sums over few rows: sums of the rows), 4-19 epilogue (four warpgroups)
constexpr uint32_t kTmemCols = 512;  // four score buffers of 128 columns
constexpr int kLse = 4;              // row tiles whose sums are held for the epilogue
constexpr int kGroup = 256;          // requests numbered at a time
constexpr float kSumTop = 0x1p60f;
enum Mode { kStats = 0, kSumsFew = 1, kSumsMany = 2, kHeld = 3, kSumsParts = 4 };  // kSumsParts: over many rows, in parts
constexpr bool many(int mode) { return mode == kSumsMany || mode == kSumsParts; }
constexpr int kHeldRows = 32;        // most rows of a request whose scores are held
constexpr int kHeldQ = 4;            // items whose queries are ahead in shared memory

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
  int q_tma;             // Q by TMA (packed rows, g <= 128), else by cp.async
  int rt;                // rows per row tile: the whole tokens of 128 rows (128 where g divides it, or is larger)
  int key_chunk;         // keys per item of the sums over few rows
  int part_tiles;        // row tiles per part of the sums over many rows
  int cluster;           // CTAs that hold one request's scores of a kv-head (0: none is held),
  int held_rows;         // of at most this many rows (16 or 32: the columns of a key tile)
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
  int b, kvh, r0, k0, steps;
  int split;         // of the keys (statistics), or part of the rows (sums over many)
  int lo[2], hi[2];  // steps in which tile t has a job (statistics, sums over many rows)
  int rt;            // row tiles (sums over few rows)
};

// Pairs of key tiles (256 keys) that the last row of part p of a request's rows
// sees some of; 0: the part has no rows.
__device__ __forceinline__ int part_pairs(const Params& prm, const Request& r, int p) {
  const long long begin = (long long)p * prm.part_tiles * prm.rt;
  const int R = r.cnt * prm.a.g;
  if (begin >= R) return 0;
  const int last = (int)((min((long long)R, begin + prm.part_tiles * prm.rt) - 1) / prm.a.g);
  return (r.P + r.first + last) / (2 * BM) + 1;
}

// Tiles of request r in this form of the kernel.
template <int MODE>
__device__ __forceinline__ int request_tiles(const Params& prm, const Request& r) {
  const WeightArgs& a = prm.a;
  const int R = r.cnt * a.g, total = r.P + r.m;
  const bool held = prm.cluster > 0 && (R == 0 || (R <= prm.held_rows && (total + BM - 1) / BM <= 512 / prm.held_rows * prm.cluster));
  if (MODE == kHeld) return held;
  if (held) return 0;
  if (MODE == kStats) return (R + 2 * prm.rt - 1) / (2 * prm.rt);
  const bool few = R <= 2 * prm.rt;
  if (MODE == kSumsFew) return few ? (total + prm.key_chunk - 1) / prm.key_chunk : 0;
  if (MODE == kSumsMany) return few ? 0 : (total + 2 * BM - 1) / (2 * BM);
  int n = 0;
  for (int p = 0; p < a.parts && !few; ++p) n += part_pairs(prm, r, p);
  return n;
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
    w.r0 = (tab.first[r + 1] - 1 - tile) * (2 * prm.rt);  // the last rows see the most keys: first
    w.k0 = w.split * a.chunk;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int row = w.r0 + t * prm.rt;
      if (row >= R) continue;
      const int end = min(w.q.P + w.q.first + (min(row + prm.rt, R) - 1) / a.g + 1, w.k0 + a.chunk);
      if (end > w.k0) w.hi[t] = (end - w.k0 + BM - 1) / BM;
    }
    w.steps = max(w.hi[0], w.hi[1]);
  } else if (MODE == kSumsFew) {
    w.k0 = at * prm.key_chunk;
    w.steps = (min(prm.key_chunk, total - w.k0) + BM - 1) / BM;
    w.rt = (R + prm.rt - 1) / prm.rt;
  } else if (many(MODE)) {
    int pair = at, begin = 0, end = R;
    if (MODE == kSumsParts) {
      w.split = a.parts - 1;  // the last rows see the most keys: first
      for (int n; pair >= (n = part_pairs(prm, w.q, w.split)) && w.split > 0; --w.split) pair -= n;
      begin = w.split * prm.part_tiles * prm.rt;
      end = min(R, begin + prm.part_tiles * prm.rt);
    }
    w.k0 = pair * (2 * BM);
    const int tok = max(0, w.k0 - w.q.P - w.q.first);  // the first counted token that sees the first key
    w.r0 = max(begin, tok * a.g / prm.rt * prm.rt);
    w.steps = tok < w.q.cnt && w.r0 < end ? (end - w.r0 + prm.rt - 1) / prm.rt : 0;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int need = max(0, w.k0 + t * BM - w.q.P - w.q.first);
      const int lo = max(0, need * a.g - w.r0) / prm.rt;
      if (w.k0 + t * BM < total && need < w.q.cnt && lo < w.steps) {
        w.lo[t] = lo;
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
  __shared__ uint64_t full[NST], empty[NST], res_full[2], res_empty[2], s_full[4], s_empty[4], drain[2];
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
      mbar_init(&empty[i], MODE == kSumsFew ? 1 : 2);  // MMA warps
      issued[i] = -1;
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&res_full[i], 1);
      mbar_init(&res_empty[i], MODE == kSumsFew ? 1 : 2);
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
    mbar_init(&drain[0], 1);
    mbar_init(&drain[1], 1);
    abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (prm.rt < BM) {  // no copy reaches the last rows of a row tile: their scores have to be numbers
    for (uint32_t at = threadIdx.x * 16; at < L::kBytes; at += kThreads * 16) *reinterpret_cast<uint4*>(smem + at) = make_uint4(0, 0, 0, 0);
    fence_async_smem();
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
  // The row tile from row r of an item (row = (counted token, head of the group)); rows
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
    for (int i = lane / CPR; i < min(prm.rt, R - r); i += STEP) {
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
  int pairs = 0;                        // key tiles of two row tiles so far (epilogue)
  bool dead = false;                    // a producer that gave up
  // The sums of an item's n row tiles for the epilogue (a whole warp).
  auto row_sums = [&](const Item& w, int n) {
    const int R = w.q.cnt * a.g;
    for (int t = 0; t < n; ++t, ++lt) {
      const int at = lt % kLse;
      float nl[BM / 32];
      int lim[BM / 32];
      const int row0 = w.r0 + t * prm.rt + lane;
      const float* lse = a.ws_lse + weight_ws_row(a, w.kvh, w.q.off, w.q.first) + row0;
#pragma unroll
      for (int e = 0; e < BM / 32; ++e) {
        const bool there = e * 32 + lane < prm.rt && row0 + e * 32 < R;
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
  };

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
        if (!many(MODE) && lane < boxes) ahead = box_page(w, x0, &bad);
        for (int j = 0; j < w.steps; ++j, ++ld) {
          const int st = ld % NST, at = j * nb & 31;
          if (!many(MODE) && at == 0) {
            pages = ahead;
            if (j * nb + 32 + lane < boxes) ahead = box_page(w, x0 + j * nb + 32, &bad);
          }
          bool go = true;
          if (lane == 0 && ld >= NST) go = wait(&empty[st], ld / NST - 1);
          dead = !__shfl_sync(0xffffffffu, (int)go, 0);
          if (dead) break;
          const uint32_t dst = sbase + L::kOffRing + st * L::kTile;
          if (lane == 0) issued[st] = ld;
          if (many(MODE)) {
            if (lane == 0 && prm.q_tma) mbar_expect_tx(&full[st], prm.rt * D * 2);
            __syncwarp();
            if (load_rows(w, w.r0 + j * prm.rt, dst, &full[st])) copies_done(&full[st]);
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
          if (lane == 0 && (many(MODE) || prm.q_tma)) mbar_expect_tx(&res_full[slot], many(MODE) ? L::kTile : prm.rt * D * 2);
          __syncwarp();
          if (many(MODE)) {
            const int x = w.k0 / prm.box_rows + t * nb + lane;
            load_keys(w, t, lane < nb ? box_page(w, x, &bad) : -1, sbase + slot * L::kTile, &res_full[slot]);
          } else if (load_rows(w, w.r0 + t * prm.rt, sbase + slot * L::kTile, &res_full[slot])) {
            copies_done(&res_full[slot]);
          }
        }
        if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(&a.status[w.b], SPEC_DEV_BAD_BLOCK);
        if (many(MODE) && !dead) row_sums(w, w.steps);
      }
    } else if (warp == 1 || (warp == 3 && MODE != kSumsFew)) {
      // ---------------------------------------------------------- MMA
      // a warp for each tile that a step multiplies, its waits (some 300 cycles each)
      // beside the other's; sums over few rows have one for both
      const int own = MODE == kSumsFew ? -1 : warp == 3 ? 1 : 0;
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
            if (own >= 0 && t != own) continue;
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
            const uint32_t n = MODE == kSumsFew ? min(BM, (R - t * prm.rt + 31) / 32 * 32) : BM;
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
    } else if (warp == 3 && MODE == kSumsFew) {
      // ---------------------------------------------------------- sums of the rows
      for (int round = 0, idx; (idx = dealt(round)) < rounds_end(n_items) && !dead; ++round) {
        if (idx >= n_items) continue;
        const Item w = find_item<MODE>(prm, tab, b0, idx, lane);
        row_sums(w, w.rt);
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
          const int row = w.r0 + g * prm.rt + r;
          const bool valid = r < prm.rt && row < R;
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
                if (e == 32) release();  // as soon as it is read
                chunk(x, vis - e);
              }
            } else {
              release();
            }
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
          const int cols = min(prm.rt, R - t * prm.rt);
          for (int j = j0; j < w.steps; j += dj) {
            const int k0 = w.k0 + j * BM, key = k0 + r;
            const float next = t == 0 && j + dj < w.steps ? old_weight(w, key + dj * BM) : 0.0f;
            float2 acc = make_float2(0.0f, 0.0f);
            const uint32_t t0 = take();
            // rows that do not see the tile's last key, or another token's rows
            const bool masked = k0 + BM - 1 > w.q.P + w.q.first || cols < prm.rt;
#pragma unroll 1
            for (int e = 0; e < cols; e += 32) {
              uint32_t x[32];
              tmem_ld32(t0 + e, x);
              tmem_wait_ld(x);
              if (e + 32 >= cols) release();  // as soon as it is read
              column_sum(x, &s_lse[at][e], &s_lim[at][e], masked, key, acc);
            }
            float sum = acc.x + acc.y;
            if (two) {  // the other row tile's share; a buffer is read before the barrier of the pair's next tile
              float* part = s_part[wg >> 1][pairs++ & 1];
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
          if (MODE == kSumsParts && w.steps == 0) continue;  // no row of the part sees a key: not added either
          const int k0 = w.k0 + g * BM, key = k0 + r;
          const float old = half == 0 && MODE == kSumsMany ? old_weight(w, key) : 0.0f;
          // rows before `edge` do not see the tile's last key
          const long long edge = (long long)(k0 + BM - 1 - w.q.P - w.q.first) * a.g;
          float2 acc = make_float2(0.0f, 0.0f);
          for (int j = 0; j < w.steps; ++j, ++lt) {
            const int at = lt % kLse;
            wait(&lse_full[at], lt / kLse);
            if (j >= lo && j < hi) {
              const int row0 = w.r0 + j * prm.rt;
              const uint32_t t0 = take();
              const bool masked = row0 < edge || row0 + prm.rt > R;
              float2 part = make_float2(0.0f, 0.0f);  // a tile's own sum: thousands of small terms would each be rounded to acc's size
#pragma unroll 1
              for (int e = half * 64; e < half * 64 + 64; e += 32) {
                uint32_t x[32];
                tmem_ld32(t0 + e, x);
                tmem_wait_ld(x);
                if (e == half * 64 + 32) release();  // as soon as it is read
                column_sum(x, &s_lse[at][e], &s_lim[at][e], masked, key, part);
              }
              acc = __fadd2_rn(acc, part);
            }
            lse_done(lt);
          }
          // the two halves of the columns, through shared memory
          if (half == 1) s_part[g][0][r] = acc.x + acc.y;
          asm volatile("bar.sync %0, 256;" ::"r"(1 + g) : "memory");
          if (half == 0) {
            const float sum = old + (acc.x + acc.y) + s_part[g][0][r];
            if (MODE == kSumsMany) put(w, key, sum);
            else if (key < w.q.P + w.q.m)
              a.ws_part[(((size_t)w.split * a.B + w.b) * a.Hkv + w.kvh) * ((size_t)a.max_prefix + a.n_max) + key] = sum;
          }
          asm volatile("bar.sync %0, 256;" ::"r"(1 + g) : "memory");
        }
      }
    }
    __syncthreads();  // the table has been read
  }

  if (MODE == kStats) asm volatile("griddepcontrol.wait;" ::: "memory");
  if ((warp == 1 || warp == 3) && elect_one()) {  // every MMA has completed before TMEM is freed
    umma_commit(&drain[warp == 3]);
    mbar_drain(&drain[warp == 3], 0);
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
// (N rows at most, 16 or 32), each CTA a run of its key tiles.  The scores of all
// tiles stay in tensor memory (N columns a tile, up to 512 / N tiles); as a tile
// arrives, each thread adds 2^x of its key to the N row sums.  The CTAs exchange their
// sums (a value per row and CTA, by st.async to every CTA of the cluster), and
// the weights come from the scores still held: K is read once.  While an item's
// sums travel the next one's tiles are loaded, multiplied and summed.
// Measured: 64 accepted paths over 256 to 16384 slots (1.19 GB) 342 us, 543 with
// the two passes; 64 single tokens 250 us; 32 requests of 8000 slots 5.2 TB/s.  It
// is bound by a cluster's own chain, 3.8 us at least for an item, and clusters of
// 8 leave 32 of 152 SMs out (15 fit).
// ---------------------------------------------------------------------------
template <int D, int N> struct HeldLayout {
  static constexpr int DH = D / 64;
  static constexpr int NST = D == 128 ? 5 : 8;
  static constexpr uint32_t kTile = BM * D * 2, kQ = N * D * 2;
  static constexpr uint32_t kOffQ = NST * kTile;
  static constexpr uint32_t kBytes = kOffQ + kHeldQ * kQ;
  static constexpr uint32_t kDyn = kBytes + 1024 < 120 * 1024 ? 120 * 1024 : kBytes + 1024;
  static_assert(kDyn + 24576 <= 227 * 1024, "dynamic and static shared memory within 227 KB");
};

// The sum (or maximum) over the warp's lanes of v[e], for lane e (and e + 16, with
// 16 of them).
template <bool MAX, int N>
__device__ __forceinline__ float warp_columns(float (&v)[N], int lane) {
#pragma unroll
  for (int o = N / 2; o; o >>= 1)
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const bool up = lane & o;
      const float give = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
      const float got = __shfl_xor_sync(0xffffffffu, give, o);
      v[i] = MAX ? fmaxf(keep, got) : keep + got;
    }
  if (N == 16) {
    const float got = __shfl_xor_sync(0xffffffffu, v[0], 16);
    v[0] = MAX ? fmaxf(v[0], got) : v[0] + got;
  }
  return v[0];
}

// N consecutive TMEM columns of this thread's lane, once they have arrived.
__device__ __forceinline__ void tmem_get(uint32_t taddr, uint32_t (&r)[32]) {
  tmem_ld32(taddr, r);
  tmem_wait_ld(r);
}
__device__ __forceinline__ void tmem_get(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]),
        "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
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

template <int D, int N>
__global__ void __launch_bounds__(kThreads, 1)
    weight_held_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ Params prm) {
  using L = HeldLayout<D, N>;
  constexpr int NST = L::NST, TILES = 512 / N, EW = 16;  // EW: epilogue warps
  const WeightArgs& a = prm.a;
  extern __shared__ uint8_t dyn_raw[];
  __shared__ uint64_t full[NST], empty[NST], q_full[kHeldQ], q_empty[kHeldQ], s_full[TILES], s_empty[TILES], drain;
  __shared__ uint64_t red_full[2], x_full[2], row_full[2], redo_full[2];
  __shared__ Table tab;
  // by item parity: each epilogue warp's row sums, each CTA's, and what the epilogue
  // needs of a row (minus log2 of its sum); s_again: the same for a second look
  __shared__ float s_red[2][EW][N], s_in[2][kHeldClusterMax][N], s_again[2][kHeldClusterMax][N], s_red2[EW][N];
  __shared__ __align__(16) float s_row[2][N];
  __shared__ __align__(16) int s_len[kGroup];
  __shared__ uint8_t s_order[kGroup];  // the group's requests, the longest first
  __shared__ int scan[kThreads / 32], abort_flag, issued[NST], s_redo[2];
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
    for (int i = 0; i < kHeldQ; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&red_full[i], EW);
      mbar_init(&x_full[i], 1);
      mbar_init(&row_full[i], 1);
      mbar_init(&redo_full[i], 1);
    }
    for (int i = 0; i < TILES; ++i) {
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
  struct HeldItem {
    Request q;
    int b, kvh, t0, nt;  // this CTA's key tiles: [t0, t0 + nt)
  };
  const int c_log2 = 31 - __clz(C);
  auto item = [&](int b0, int idx) {
    HeldItem w;
    const int r = s_order[idx / a.Hkv];
    w.kvh = idx % a.Hkv;
    w.b = b0 + r;
    w.q = tab.r[r];
    const int tiles = (w.q.P + w.q.m + BM - 1) / BM, each = (tiles + C - 1) >> c_log2;
    w.t0 = rank * each;
    w.nt = max(0, min(each, tiles - w.t0));
    return w;
  };
  // the first round from `round` on that deals this cluster an item, -1: none is left
  auto next_item = [&](int& round, int n) -> int {
    for (;; ++round) {
      const int idx = dealt(round);
      if (idx < n) return idx;
      if (idx >= rounds_end(n)) return -1;
    }
  };

  int ld = 0;     // key tiles of this CTA so far (stream, MMA, epilogue)
  int units = 0;  // items with tiles here (Q, MMA), items with rows (sums, epilogue)
  int looks = 0;  // exchanges of second looks (epilogue)
  bool dead = false;
  for (int b0 = 0; b0 < a.B; b0 += kGroup) {
    const int n_requests = build_table<kHeld>(prm, tab, b0, scan), n_items = n_requests * a.Hkv;
    {  // the longest first: the shares of the clusters come out alike
      const int c = threadIdx.x;
      const bool in = c < kGroup && tab.first[c + 1] > tab.first[c];
      if (c < kGroup) s_len[c] = in ? tab.r[c].P + tab.r[c].m : -1;
      __syncthreads();
      if (in) {
        const int mine = s_len[c];
        const int there = min(kGroup, a.B - b0);
        int before = 0;
#pragma unroll 4
        for (int j = 0; j < there; j += 4) {
          const int4 x = *reinterpret_cast<const int4*>(&s_len[j]);
          before += x.x > mine || (x.x == mine && j < c);
          before += x.y > mine || (x.y == mine && j + 1 < c);
          before += x.z > mine || (x.z == mine && j + 2 < c);
          before += x.w > mine || (x.w == mine && j + 3 < c);
        }
        s_order[before] = (uint8_t)c;
      }
      __syncthreads();
    }
    if (warp == 0) {
      // ---------------------------------------------------------- K
      const int nb = BM / prm.box_rows;
      // the page of box x of an item (boxes count from the request's slot 0), -1 behind
      // its keys, -2 at a bad id
      auto page_of = [&](const HeldItem& w, int x) -> int {
        const int k = x * prm.box_rows;
        if (k >= w.q.P + w.q.m) return -1;
        const int page = __ldg(a.block_table + (size_t)w.b * a.max_blocks + (k >> prm.bs_log2));
        return page >= 0 && page < a.num_blocks ? page : -2;
      };
      // the first pages of the next item are looked up before this one's tiles go out
      int round = 0, idx = next_item(round, n_items), first_pages = -1;
      HeldItem w = {};
      auto look = [&]() {
        if (idx < 0) return;
        w = item(b0, idx);
        first_pages = w.q.cnt > 0 && lane < w.nt * nb ? page_of(w, w.t0 * nb + lane) : -1;
      };
      look();
      while (idx >= 0 && !dead) {
        const HeldItem v = w;
        int ahead = first_pages, pages = -1;
        bool bad = false;
        ++round;
        idx = next_item(round, n_items);
        look();
        for (int j = 0; j < v.nt && v.q.cnt > 0; ++j, ++ld) {
          const int st = ld % NST, at = j * nb & 31;
          if (at == 0) {
            pages = ahead;
            bad |= pages == -2;
            if (j * nb + 32 + lane < v.nt * nb) ahead = page_of(v, v.t0 * nb + j * nb + 32 + lane);
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
            const int k = (v.t0 + j) * BM + lane * prm.box_rows;
            const int y = page < 0 ? (int)prm.rows_total : ((page * a.Hkv + v.kvh) << prm.bs_log2) + (k & (a.block_size - 1));
#pragma unroll
            for (int h = 0; h < L::DH; ++h)
              tma_load_2d(sbase + st * L::kTile + h * (BM * 128) + lane * prm.box_rows * 128, &tmap_k, h * 64, y, &full[st]);
          }
        }
        if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(&a.status[v.b], SPEC_DEV_BAD_BLOCK);
      }
    } else if (warp == 2) {
      // ---------------------------------------------------------- Q: 32 rows, zeros behind the item's
      // An item is announced once the next one's copies are out.
      constexpr int CPR = D / 8, STEP = 32 / CPR;
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q);
      const int ch = lane % CPR;
      int round = 0, idx = next_item(round, n_items), pending = -1;
      HeldItem w = {};
      int token = 0;  // row of q of counted token `lane`, looked up an item ahead
      auto look = [&]() {
        if (idx < 0) return;
        w = item(b0, idx);
        token = w.q.off + (lane >= w.q.cnt ? 0 : a.path ? a.path[(size_t)w.b * a.path_stride + w.q.first + lane] : w.q.first + lane);
      };
      auto announce = [&]() {
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[pending]);
      };
      look();
      while (idx >= 0 && !dead) {
        const HeldItem v = w;
        const int tokens = token;
        ++round;
        idx = next_item(round, n_items);
        look();
        if (v.q.cnt == 0 || v.nt == 0) continue;
        const int slot = units % kHeldQ, R = v.q.cnt * a.g;
        bool go = true;
        if (lane == 0 && units >= kHeldQ) go = wait(&q_empty[slot], units / kHeldQ - 1);
        dead = !__shfl_sync(0xffffffffu, (int)go, 0);
        if (dead) break;
        const uint32_t dst = L::kOffQ + slot * L::kQ + (ch >> 3) * (N * 128);
#pragma unroll
        for (int i0 = 0; i0 < N; i0 += STEP) {
          const int i = i0 + lane / CPR, tok = min(i / a.g, 31);
          const size_t row = __shfl_sync(0xffffffffu, tokens, tok);
          const uint32_t at = dst + i * 128 + (((ch & 7) ^ (i & 7)) << 4);
          if (i < R) cp_async16(sbase + at, q + (row * a.Hq + v.kvh * a.g + i % a.g) * D + ch * 8);
          else *reinterpret_cast<uint4*>(smem + at) = make_uint4(0, 0, 0, 0);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (pending >= 0) {
          asm volatile("cp.async.wait_group 1;" ::: "memory");
          announce();
        }
        pending = slot;
        ++units;
      }
      cp_async_wait();
      if (pending >= 0) announce();
    } else if (warp == 1) {
      // ---------------------------------------------------------- MMA: A = K tile, B = Q
      const uint64_t ring = smem_desc_sw128(sbase, 16, 1024), qd0 = smem_desc_sw128(sbase + L::kOffQ, 16, 1024);
      constexpr uint32_t idesc = idesc_bf16(N, 0);
      const bool leader = elect_one();
      for (int round = 0, idx; (idx = next_item(round, n_items)) >= 0; ++round) {
        const HeldItem w = item(b0, idx);
        if (w.q.cnt == 0 || w.nt == 0) continue;
        wait(&q_full[units % kHeldQ], units / kHeldQ);
        const uint64_t qd = qd0 + (uint64_t)((units % kHeldQ) * (L::kQ >> 4));
        for (int j = 0; j < w.nt; ++j, ++ld) {
          const int st = ld % NST, s = ld % TILES;
          wait(&full[st], ld / NST);
          if (ld >= TILES) wait(&s_empty[s], ld / TILES - 1);
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
        if (leader) umma_commit(&q_empty[units % kHeldQ]);
        __syncwarp();
        ++units;
      }
    } else if (warp == 3) {
      // ---------------------------------------------------------- row sums over the cluster (row = lane)
      // Item k + 1's sums leave after item k's have come in from every CTA, so two
      // buffers do.
      for (int round = 0, idx; (idx = next_item(round, n_items)) >= 0; ++round) {
        const HeldItem w = item(b0, idx);
        if (w.q.cnt == 0) continue;
        const int buf = units & 1, phase = units >> 1;
        wait(&red_full[buf], phase);
        const bool row = lane < N;
        float v = row ? s_red[buf][0][lane] : 0.0f;
#pragma unroll
        for (int k = 1; k < EW; ++k) v += row ? s_red[buf][k][lane] : 0.0f;
        if (lane == 0) mbar_expect_tx(&x_full[buf], C * N * 4);
        __syncwarp();
        for (int k = 0; k < C && row; ++k) send_async(&s_in[buf][rank][lane], &x_full[buf], k, v);
        __syncwarp();
        mbar_wait_cluster(&x_full[buf], phase & 1, &abort_flag);
        float sum = 0.0f;
        for (int k = 0; k < C && row; ++k) sum += s_in[buf][k][lane];
        const bool there = lane < w.q.cnt * a.g, fits = !there || (sum >= 1.0f / kSumTop && sum < kSumTop);
        if (row) s_row[buf][lane] = there ? -log2f(sum) : -INFINITY;
        const bool redo = !__all_sync(0xffffffffu, fits);
        if (lane == 0) s_redo[buf] = redo;
        __syncwarp();
        if (lane == 0) mbar_arrive(&row_full[buf]);
        ++units;
      }
    } else if (warp >= 4) {
      // ---------------------------------------------------------- epilogue
      // Item k + 1's scores are summed while item k's sums travel, as long as tensor
      // memory holds both.
      const int ew = warp - 4, wg = ew >> 2, quad = warp & 3, r = quad * 32 + lane;
      const uint32_t tS = tmem + ((uint32_t)(quad * 32) << 16);
      const float c2 = a.scale_log2;
      auto all_sync = [&]() { asm volatile("bar.sync 1, 512;" ::: "memory"); };
      // Scores of key tile t0 + j (the CTA's tile number n), -inf where row `e`, whose
      // last visible slot lane e holds in `lim`, does not see the key.
      auto tile = [&](const HeldItem& w, int j, int n, float (&x)[N]) {
        uint32_t u[N];
        tmem_get(tS + (uint32_t)(n % TILES) * N, u);
        const int k0 = (w.t0 + j) * BM;
        if (k0 + BM - 1 > w.q.P + w.q.first) {
          const int lim = lane < w.q.cnt * a.g ? w.q.P + w.q.first + lane / a.g : -1;
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
      // A row's value over the cluster for a second look: the CTA's warps meet, warp 4
      // does what warp 3 does for the first look.  In warp 4 the result of row `lane`.
      auto exchange = [&](float v, bool max) -> float {
        if (lane < N) s_red2[ew][lane] = v;
        all_sync();
        const int buf = looks & 1, phase = looks >> 1;
        ++looks;
        if (ew != 0) return 0.0f;
        const bool row = lane < N;
        for (int k = 1; k < EW && row; ++k) v = max ? fmaxf(v, s_red2[k][lane]) : v + s_red2[k][lane];
        __syncwarp();
        if (lane == 0) mbar_expect_tx(&redo_full[buf], C * N * 4);
        __syncwarp();
        for (int k = 0; k < C && row; ++k) send_async(&s_again[buf][rank][lane], &redo_full[buf], k, v);
        __syncwarp();
        mbar_wait_cluster(&redo_full[buf], phase & 1, &abort_flag);
        float all = max ? -INFINITY : 0.0f;
        for (int k = 0; k < C && row; ++k) all = max ? fmaxf(all, s_again[buf][k][lane]) : all + s_again[buf][k][lane];
        return all;
      };
      auto old_weight = [&](const HeldItem& w, int j) -> float {
        const int key = (w.t0 + j) * BM + r;
        return a.before && j < w.nt && key < w.q.P ? a.decay * a.before[((size_t)w.b * a.Hkv + w.kvh) * a.stride + key] : 0.0f;
      };
      auto put = [&](const HeldItem& w, int j, float sum) {
        const int key = (w.t0 + j) * BM + r;
        if (key < w.q.P + w.q.m && !w.q.quiet) a.weight[((size_t)w.b * a.Hkv + w.kvh) * a.stride + key] = sum;
      };
      // the weights of item `idx`, the k-th with rows, whose first tile here was number
      // n0; old: what its first key of this thread had
      auto finish = [&](int idx, int k, int n0, float old) {
        const HeldItem w = item(b0, idx);
        const int nt = w.nt, buf = k & 1;
        wait(&row_full[buf], k >> 1);
        if (s_redo[buf]) {  // a sum left fp32's middle: against the rows' maxima
          const int R = w.q.cnt * a.g;
          float acc[N];
#pragma unroll
          for (int e = 0; e < N; ++e) acc[e] = -INFINITY;
          for (int j = wg; j < nt; j += 4) {
            float x[N];
            tile(w, j, n0 + j, x);
#pragma unroll
            for (int e = 0; e < N; ++e) acc[e] = fmaxf(acc[e], x[e]);
          }
          float top = exchange(warp_columns<true, N>(acc, lane), true);
          top = lane < R && top > -INFINITY ? top * c2 : 0.0f;
          if (ew == 0 && lane < N) s_row[buf][lane] = top;
          all_sync();
#pragma unroll
          for (int e = 0; e < N; ++e) acc[e] = 0.0f;
          for (int j = wg; j < nt; j += 4) {
            float x[N];
            tile(w, j, n0 + j, x);
#pragma unroll
            for (int e = 0; e < N; ++e) acc[e] += fast_exp2(fmaf(x[e], c2, -s_row[buf][e]));
          }
          const float sum = exchange(warp_columns<false, N>(acc, lane), false);
          if (ew == 0 && lane < N) s_row[buf][lane] = lane < R ? -(top + log2f(sum)) : -INFINITY;
          all_sync();
        }
        for (int j = wg; j < nt; j += 4) {
          const float next = old_weight(w, j + 4);
          float x[N];
          tile(w, j, n0 + j, x);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_empty[(n0 + j) % TILES]);
          float2 p = make_float2(0.0f, 0.0f);
#pragma unroll
          for (int e = 0; e < N; e += 4) {
            const float4 n4 = *reinterpret_cast<const float4*>(&s_row[buf][e]);
            p.x += fast_exp2(fmaf(x[e], c2, n4.x)) + fast_exp2(fmaf(x[e + 1], c2, n4.y));
            p.y += fast_exp2(fmaf(x[e + 2], c2, n4.z)) + fast_exp2(fmaf(x[e + 3], c2, n4.w));
          }
          put(w, j, old + (p.x + p.y));
          old = next;
        }
      };
      // One turn: sums of the next item (if tensor memory has room beside the one
      // whose weights are due), then the weights that are due.
      int late = -1, late_n0 = 0;  // the item whose weights are due, and its first tile
      float late_old = 0.0f;
      for (int round = 0;;) {
        const int idx = next_item(round, n_items);
        const bool more = idx >= 0;
        HeldItem w = {};
        if (more) {
          w = item(b0, idx);
          if (w.q.cnt == 0) {  // no rows: the old weights alone
            for (int j = wg; j < w.nt; j += 4) put(w, j, old_weight(w, j));
            ++round;
            continue;
          }
        }
        const int nt = w.nt;
        const float old = more ? old_weight(w, wg) : 0.0f;
        const bool room = more && (late < 0 || ld + nt - late_n0 <= TILES);
        if (room) {
          float acc[N];
#pragma unroll
          for (int e = 0; e < N; ++e) acc[e] = 0.0f;
          for (int j = wg; j < nt; j += 4) {
            wait(&s_full[(ld + j) % TILES], (ld + j) / TILES);
            tc_fence_after();
            float x[N];
            tile(w, j, ld + j, x);
#pragma unroll
            for (int e = 0; e < N; ++e) acc[e] += fast_exp2(x[e] * c2);
          }
          const float mine = warp_columns<false, N>(acc, lane);
          if (lane < N) s_red[units & 1][ew][lane] = mine;
          __syncwarp();
          if (lane == 0) mbar_arrive(&red_full[units & 1]);
        }
        if (late >= 0) finish(late, units - 1, late_n0, late_old);
        late = -1;
        if (room) {
          late = idx;
          late_n0 = ld;
          late_old = old;
          ld += nt;
          ++units;
          ++round;
        } else if (!more) {
          break;
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
// of its keys left: 8 lanes a row, 32 rows a CTA.  a.per_req counts these tiles.
constexpr int kJoinThreads = 256, kJoinRows = kJoinThreads / 8;
__global__ void __launch_bounds__(kJoinThreads) weight_join_kernel(const WeightArgs a, int tiles) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tile = blockIdx.x % tiles, kvh = blockIdx.x / tiles;
  int b, at_tile;  // the division in 32 bits: 8192 CTAs of a prompt's rows pay for it
  if (a.per_req > 0) {
    b = tile / a.per_req;
    at_tile = tile - b * a.per_req;
  } else {
    b = weight_find(a, tile, kJoinRows);
    at_tile = (int)max(-1LL, tile - weight_first_tile(a, b, kJoinRows));
  }
  WeightRequest r;
  const bool bad = weight_check(a, b, r) != 0 || at_tile < 0 || at_tile > (r.cnt * a.g - 1) / kJoinRows || r.cnt == 0;
  const int row = at_tile * kJoinRows + threadIdx.x / 8, part = threadIdx.x % 8;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (bad) return;
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

// The parts of a request's rows added up, in their order: a thread a key.
constexpr int kAddThreads = 256;
__global__ void __launch_bounds__(kAddThreads) weight_add_kernel(const __grid_constant__ Params prm, int pairs) {
  const WeightArgs& a = prm.a;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int kvh = blockIdx.x % a.Hkv, pair = blockIdx.x / a.Hkv % pairs, b = blockIdx.x / a.Hkv / pairs;
  WeightRequest r;
  if (weight_check(a, b, r) || a.status[b] != 0 || r.cnt * a.g <= 2 * prm.rt) return;
  const int key = pair * kAddThreads + threadIdx.x;
  if (key >= r.P + r.m) return;
  const Request q = {r.off, r.m - r.cnt, r.cnt, r.P, r.m, 0};
  const size_t at = ((size_t)b * a.Hkv + kvh) * a.stride + key;
  float sum = a.before && key < r.P ? a.decay * a.before[at] : 0.0f;
  for (int p = 0; p < a.parts; ++p) {
    if (pair < part_pairs(prm, q, p))
      sum += a.ws_part[(((size_t)p * a.B + b) * a.Hkv + kvh) * ((size_t)a.max_prefix + a.n_max) + key];
  }
  a.weight[at] = sum;
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

template <int D, int N>
static void held_config(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr, int c) {
  cfg.gridDim = dim3(c, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = HeldLayout<D, N>::kDyn;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = c;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
}

// Clusters of c CTAs that device `dev` (the current one) runs at once; asked for
// once per device and size.
template <int D, int N>
static int held_clusters(int dev, int c) {
  static std::atomic<int> known[64][kHeldClusterMax + 1];  // number + 1
  const bool keep = dev < 64;
  if (keep && known[dev][c] > 0) return known[dev][c] - 1;
  int n = 0;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  held_config<D, N>(cfg, attr, c);
  if (cudaFuncSetAttribute(weight_held_kernel<D, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)HeldLayout<D, N>::kDyn) != cudaSuccess ||
      cudaFuncSetAttribute(weight_held_kernel<D, N>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, weight_held_kernel<D, N>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  if (keep) known[dev][c] = n + 1;
  return n;
}

template <int D, int N>
static cudaError_t launch_held(const CUtensorMap& mk, const Params& prm, int fit, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  held_config<D, N>(cfg, attr, prm.cluster);
  cfg.gridDim = dim3((unsigned)(std::min<long long>(fit, (long long)prm.a.B * prm.a.Hkv) * prm.cluster), 1, 1);
  cfg.stream = stream;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, weight_held_kernel<D, N>, mk, prm);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// CTAs per cluster, by a model of what one request's kv-head costs a cluster: some
// 3.8 us at least (the exchange), 0.9 us a key tile where two items' scores fit
// beside each other, else 3.3 us and 0.7 us a tile.  Measured with 512 of them of
// 4000 keys each in clusters of 2, 4, 8 and 16 (76, 36, 15 and 7 fit on the GPU): 120, 118, 146 and
// 271 us; of 8000 keys in 4, 8 and 16: 221, 206 and 287; 1024 of 1000 keys in 1, 2,
// 4: 71, 80, 139.  Two passes over K (385 us for the 512 of 8000 keys) are the
// other way.  The costs are those of D 128; D 64 is charged the same, and its two
// passes by their bytes, less than they take.  At D 64, 32/8 heads, L2 flushed, two
// passes and clusters of 2, 4, 8 (* the choice): 64 requests of 4 rows over 4000 slots
// 188, 91*, 97, 122 us, over 8000 355, 171*, 175, 205; of 32 rows over 4000 186, 95*,
// 103, 136, but over 8000 350*, -, 181, 217 and over 16000 663*, -, -, 396: there the
// held form would take little more than half.
// Nodes that a path leaves out have no key, so its tree does not count as keys.
// Returns the clusters that fit, 0: no request is held.
template <int D, int N>
static int held_plan(const WeightArgs& a, int dev, int* cluster) {
  constexpr int kMost = 512 / N;  // key tiles of a CTA
  const long long keys = std::max(1LL, (long long)a.max_prefix + (a.path ? 0 : a.n_max));
  const long long tiles = (keys + BM - 1) / BM, units = (long long)a.B * a.Hkv;
  double best = 25.0 + 2.0 * units * keys * D * 2 / 5.7e6;  // us
  int fits = 0;
  // packed rows: not for a batch whose requests have more on average
  const long long average = a.window > 0 ? std::min<long long>(a.window, a.T / a.B) : a.T / a.B;
  if (a.g > N || (!a.path && average * a.g > 2 * N)) return 0;
  for (int c = 1; c <= kHeldClusterMax; c *= 2) {
    const long long nt = (tiles + c - 1) / c;
    if (nt > kMost) continue;
    const int fit = held_clusters<D, N>(dev, c);
    if (fit == 0) continue;
    const double cost = (double)((units + fit - 1) / fit) * std::max(3.8, nt <= kMost / 2 ? 0.9 * nt : 3.3 + 0.7 * nt);
    if (cost >= best) continue;
    best = cost;
    fits = fit;
    *cluster = c;
  }
  return fits;
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
  prm.q_tma = !a.path && a.g <= BM && a.T > 0;
  prm.rt = a.g <= BM ? BM / a.g * a.g : BM;
  // sums over few rows: some two items for every CTA, of 256 to 2048 keys
  const long long keys = ((long long)a.max_prefix + a.n_max) * a.B * a.Hkv / (2LL * sms);
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
  prm.part_tiles = (int)std::max(1LL, ((rows + prm.rt - 1) / prm.rt + a.parts - 1) / a.parts);
  // Scores are held where a request has few rows; one with more rows, or more keys
  // than its cluster holds, goes the other way, inside the kernels.
  bool first = true;
  const long long longest = (long long)a.max_prefix + a.n_max;
  prm.held_rows = rows <= 16 ? 16 : kHeldRows;
  const int fit = prm.held_rows == 16 ? held_plan<D, 16>(a, dev, &prm.cluster) : held_plan<D, 32>(a, dev, &prm.cluster);
  if (fit > 0) {
    e = prm.held_rows == 16 ? launch_held<D, 16>(mk, prm, fit, stream) : launch_held<D, 32>(mk, prm, fit, stream);
    if (e != cudaSuccess) return e;
    if (rows <= prm.held_rows && longest <= 512LL / prm.held_rows * prm.cluster * BM) return cudaSuccess;  // every request's are held
    first = false;
  }
  const int dyn = (int)Layout<D>::kDyn;
  if (rows > 0) {
    // n_max may be far above what a batch has: the fewer of each request's most and
    // the packing's tiles (as the row tiles of the fp32 kernels)
    WeightArgs join = a;
    const long long each = (rows + kJoinRows - 1) / kJoinRows, packed = (long long)a.T * a.g / kJoinRows + a.B;
    join.per_req = each * a.B < packed ? (int)each : 0;
    const int tiles = (int)std::min(each * a.B, packed);
    e = launch(weight_tc_kernel<D, kStats>, sms, kThreads, dyn, first, stream, mk, mq, prm);
    if (e == cudaSuccess) e = launch(weight_join_kernel, (long long)tiles * a.Hkv, kJoinThreads, 0, false, stream, join, tiles);
  }
  if (e == cudaSuccess) e = launch(weight_tc_kernel<D, kSumsFew>, sms, kThreads, dyn, first && rows == 0, stream, mk, mq, prm);
  if (e == cudaSuccess && rows > 2 * prm.rt) {
    if (a.parts == 1) return launch(weight_tc_kernel<D, kSumsMany>, sms, kThreads, dyn, false, stream, mk, mq, prm);
    e = launch(weight_tc_kernel<D, kSumsParts>, sms, kThreads, dyn, false, stream, mk, mq, prm);
    if (e == cudaSuccess) {
      const int pairs = (int)((longest + kAddThreads - 1) / kAddThreads);
      e = launch(weight_add_kernel, (long long)pairs * a.Hkv * a.B, kAddThreads, 0, false, stream, prm, pairs);
    }
  }
  return e;
}

}  // namespace wtc

cudaError_t launch_weight_tc(const WeightArgs& a, cudaStream_t stream) {
  return a.D == 64 ? wtc::launch_d<64>(a, stream) : wtc::launch_d<128>(a, stream);
}

}  // namespace spectree
