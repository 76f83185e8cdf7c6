// Prompt attention on the 5th-generation tensor cores (tcgen05), bf16 inputs,
// fp32 scores and accumulators in tensor memory.
//
// Per work item (256 rows of one request's kv-head group, one key range) a CTA
// holds two 128-row tiles t = 0, 1 and walks the keys 128 at a time:
//   S_t = Q_t K_j^T          A = Q (shared memory), B = K tile (shared memory)
//   P_t = 2^(S_t c - m)      softmax warps, row r == TMEM lane r, one thread per
//                            row; bf16 P over the S columns just read
//   O_t += P_t V_j           A = P (tensor memory), B = V tile (shared memory)
// The two tiles share every K and V stage, and while one tile's scores are in
// the softmax the tensor core works for the other:
//   ... PV_j(0) QK_{j+1}(0) | PV_j(1) QK_{j+1}(1) | PV_{j+1}(0) ...
// Each tile's MMAs are issued by a warp of its own (a wait behind issued MMAs
// returns only once the tensor core has taken them, and the other tile's are
// then already queued).  They complete in the order of issue, so S_t may be
// overwritten right after PV_j(t) without a wait.  The two warps take turns,
// PV and QK of a step at a time: left alone they fall in step, both tiles'
// MMAs at one time and both tiles' softmaxes at another.
//
// Reference m of a row: softmax(x) = 2^(xc - m) / sum 2^(xc - m) for ANY m, and
// fp32 and bf16 hold 2^127.  So m starts at 0 and no maximum is taken, as long
// as the sum of 64 weights stays below 2^30 and the first visible ones reach
// 2^-30.  Otherwise that half tile is done again against its own maximum, and O
// and the sum are scaled to it.  What the weights take of fp32's range is lost
// to V: magnitudes of 2^-60 to 2^80 neither overflow (2^30 of 64 weights, 2^18
// keys and more) nor lose bits below 2^-126 (2^-36 of the largest weight, 24
// bits).  Limits of 2^60, 2^30 and 2^20 cost the same where scores have a
// deviation of 1 (natural units) and nearly so at 3; at 10 one prompt of 16384
// took 1330, 1410 and 1637 us, a redo for every larger maximum.
//
// What bounds it, and what it measured (32/8 heads, D 128, one GB300):
//   long prompts: the tensor core.  A step of 2 x 128 x 128 takes 2048 cycles of
//   it, and shared memory is as busy (Q and K of a QK come from it).  One prompt
//   of 16384 tokens: 1320 us on a cold GPU (1666 TFLOP/s, 0.87 of the measured
//   bf16 burst), 1435 us one after another at the power cap (0.90 of the
//   sustained rate).  With sums of unrounded weights 1258 us, and of these 126
//   for the exponentials.
//   prompts of some 500 tokens: the few steps of an item against its change
//   (first step, output rows, next Q), about 10 kcycles each way.
//   single tokens over long prefixes: HBM, 5.6 TB/s on 64 requests cold, 5.8 one
//   after another.
#include <algorithm>

#include "prompt.cuh"
#include "tcgen05.cuh"

namespace spectree {

namespace ptc {

using namespace tc5;

constexpr int BM = 128;              // rows per tile (M of the MMA)
constexpr int BN = 128;              // keys per step
constexpr int kRows = kPromptTcRows; // rows per work item
constexpr int HC = BN / 2;           // keys per softmax half
constexpr int kThreads = 384;        // warps: 0 K loads, 1 and 3 MMA of tiles 0 and 1, 2 work items, Q and V loads, 4-7 softmax of tile 0, 8-11 of tile 1
constexpr uint32_t kTmemCols = 512;  // S_0, S_1 at 0, 128; O_0, O_1 at 256, 384
constexpr float kSumLimit = 1073741824.0f;  // 2^30
constexpr int kOrderMax = 256;       // batches up to this size run longest request first
static_assert(kRows == 2 * BM, "two row tiles per item");

template <int D> struct Layout {
  static constexpr int DH = D / 64;            // 128-byte halves of a row
  static constexpr int NST = D == 128 ? 5 : 8; // stages of the ring that K and V tiles share
  static constexpr uint32_t kTile = BM * D * 2;   // one Q tile, one K or V stage
  static constexpr uint32_t kOffKV = 2 * kTile;
  static constexpr uint32_t kBytes = kOffKV + NST * kTile;
  static constexpr uint32_t kDyn = kBytes + 1024 < 120 * 1024 ? 120 * 1024 : kBytes + 1024;  // one CTA per SM (all of TMEM)
  static_assert(kDyn + 2048 <= 227 * 1024, "dynamic and (below 2 KB) static shared memory within 227 KB");
};

struct Params {
  PromptArgs a;
  long long rows_total;  // num_blocks * Hkv * block_size: rows of the 2-D cache view
  int box_rows;          // rows per TMA box: min(block_size, 128)
  int bs_log2;           // block_size = 1 << bs_log2
  int q_tma;             // Q by TMA (g divides 128), else by cp.async
};

// One work item; valid = 0 ends every role's loop.
struct Work {
  int valid, b, off, n, P, kvh, r0, split, k_begin;
  int nt[2];  // key steps of the two row tiles (0: the tile has no rows or sees none of the keys)
};

// The requests in decreasing key count (ties by index), with the number of row
// tiles before each: the longest items start first.  Only the requests' own
// arguments count here, so every CTA numbers the items alike.
struct Order {
  int first[kOrderMax + 1];
  uint8_t req[kOrderMax];
};

__device__ __forceinline__ int row_tiles(const PromptArgs& a, int off, int n, int P) {
  return prompt_check(a, off, n, P) ? 0 : (int)(((long long)n * a.g + kRows - 1) / kRows);
}

__device__ __forceinline__ void order_requests(const PromptArgs& a, Order& o, int* len, int* tiles) {
  const int c = threadIdx.x;
  if (c < a.B) {
    const int off = a.seq_off[c], n = a.seq_off[c + 1] - off, P = a.prefix_len[c];
    tiles[c] = row_tiles(a, off, n, P);
    len[c] = tiles[c] ? P + n : 0;
  }
  __syncthreads();
  if (c < a.B) {
    int rank = 0, before = 0;
    for (int j = 0; j < a.B; ++j) {
      const bool ahead = len[j] > len[c] || (len[j] == len[c] && j < c);
      rank += ahead;
      before += ahead ? tiles[j] : 0;
    }
    o.req[rank] = (uint8_t)c;
    o.first[rank] = before;
    if (rank == a.B - 1) o.first[a.B] = before + tiles[c];
  }
  __syncthreads();
}

// Work item `idx` (one warp, all lanes get it); valid = 0 when it is empty.
__device__ __forceinline__ Work find_work(const Params& prm, const Order& o, uint32_t idx, int lane) {
  const PromptArgs& a = prm.a;
  Work w = {};
  w.split = (int)(idx % (uint32_t)a.splits);
  idx /= (uint32_t)a.splits;
  w.kvh = (int)(idx % (uint32_t)a.Hkv);
  const int tile = (int)(idx / (uint32_t)a.Hkv);
  int b, mt;
  if (a.B <= kOrderMax) {
    if (tile >= o.first[a.B]) return w;
    int cnt = 0;  // requests whose first tile is not above this one (empty ones rank last)
    for (int r = lane; r < a.B; r += 32) cnt += o.first[r] <= tile;
    cnt = warp_sum_i(cnt);
    const int r = cnt - 1;
    b = o.req[r];
    mt = o.first[r + 1] - 1 - tile;  // the last rows see the most keys: first
  } else {
    int lo = 0, hi = a.B;  // first_tile(lo) <= tile < first_tile(hi), 32 probes a round
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32;
      const int at = lo + lane * step;
      const bool below = at < hi && prompt_first_tile(a, at, kRows) <= tile;
      const int last = __popc(__ballot_sync(0xffffffffu, below)) - 1;  // lane 0 is always below
      const int nlo = lo + max(last, 0) * step;
      hi = min(hi, nlo + step);
      lo = nlo;
    }
    b = lo;
    const long long at = tile - prompt_first_tile(a, b, kRows);
    if (at < 0 || at > (1 << 30)) return w;
    mt = (int)at;
  }
  PromptRequest rq;
  if (lane == 0) rq = prompt_request(a, b);
  rq.off = __shfl_sync(0xffffffffu, rq.off, 0);
  rq.n = __shfl_sync(0xffffffffu, rq.n, 0);
  rq.P = __shfl_sync(0xffffffffu, rq.P, 0);
  const bool ok = __shfl_sync(0xffffffffu, (int)rq.ok, 0);
  const int R = rq.n * a.g;  // < 2^30
  if (!ok || mt >= (1 << 22) || mt * kRows >= R) return w;
  w.b = b;
  w.off = rq.off;
  w.n = rq.n;
  w.P = rq.P;
  w.r0 = mt * kRows;
  w.k_begin = w.split * a.chunk;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int first = w.r0 + t * BM;
    if (first >= R) continue;
    const int end = min(rq.P + (min(first + BM, R) - 1) / a.g + 1, w.k_begin + a.chunk);
    if (end > w.k_begin) w.nt[t] = (end - w.k_begin + BN - 1) / BN;
  }
  w.valid = w.nt[0] > 0 || w.nt[1] > 0;
  return w;
}

// Row of the 2-D cache view where the box starting at key k of the item's
// kv-head begins; keys past the request, or at a bad block id, read the
// out-of-range row `rows_total` (zero fill).
__device__ __forceinline__ int box_row(const Params& prm, const int32_t* bt, int kvh, int k, int Lk, int* bad) {
  const PromptArgs& a = prm.a;
  int y = (int)prm.rows_total;
  if (k < Lk) {
    const int blk = __ldg(bt + (k >> prm.bs_log2));
    if (blk >= 0 && blk < a.num_blocks) y = ((blk * a.Hkv + kvh) << prm.bs_log2) + (k & (a.block_size - 1));  // < rows_total
    else *bad = 1;
  }
  return y;
}

// 4 x 4 transpose among four neighbouring lanes: afterwards u[s] of lane i is
// what u[i] of lane s was.
__device__ __forceinline__ void transpose4(uint4 (&u)[4], int lane) {
  auto swap = [&](uint4& a, uint4& b, int d) {  // lanes with bit d send a, the others b
    const bool hi = lane & d;
    uint4 x = hi ? a : b;
    x.x = __shfl_xor_sync(0xffffffffu, x.x, d);
    x.y = __shfl_xor_sync(0xffffffffu, x.y, d);
    x.z = __shfl_xor_sync(0xffffffffu, x.z, d);
    x.w = __shfl_xor_sync(0xffffffffu, x.w, d);
    if (hi) a = x;
    else b = x;
  };
  swap(u[0], u[1], 1);
  swap(u[2], u[3], 1);
  swap(u[0], u[2], 2);
  swap(u[1], u[3], 2);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_tc_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                     const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ Params prm) {
  using L = Layout<D>;
  constexpr int NST = L::NST;
  const PromptArgs& a = prm.a;
  extern __shared__ uint8_t dyn_raw[];
  __shared__ uint64_t kv_full[NST], kv_empty[NST], s_full[2], p_full[2][2], o_done[2][2], q_full, q_empty, w_full[2],
      w_empty[2], turn[2], drain[2], next_full;
  __shared__ __align__(16) uint4 next_cta[1];
  __shared__ Work work[2];
  __shared__ Order order;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag, kv_issued[NST], q_issued;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn_raw) + 1023) & ~(uintptr_t)1023);
  const uint32_t sbase = smem_u32(smem);
  if (threadIdx.x == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(&kv_full[i], 1);
      kv_issued[i] = -1;
      mbar_init(&kv_empty[i], 2);  // both MMA warps
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[t][0], 4);
      mbar_init(&p_full[t][1], 4);
      mbar_init(&o_done[t][0], 1);
      mbar_init(&o_done[t][1], 1);
      mbar_init(&w_full[t], 1);
      mbar_init(&w_empty[t], 11);  // K/V warp, two MMA warps, eight softmax warps
    }
    mbar_init(&q_full, 1);
    mbar_init(&q_empty, 2);
    mbar_init(&next_full, 1);
    mbar_init(&turn[0], 1);
    mbar_init(&turn[1], 1);
    mbar_init(&drain[0], 1);
    mbar_init(&drain[1], 1);
    abort_flag = 0;
    q_issued = -1;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (a.B <= kOrderMax) {
    // scratch of the ranking: the K/V ring's room, which no copy has reached yet
    int* scratch = reinterpret_cast<int*>(smem + L::kOffKV);
    order_requests(a, order, scratch, scratch + kOrderMax);
    fence_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  // The waits of the MMA and softmax warps.  Every lane polls, and nothing
  // branches on the outcome: a wait that runs out sets the abort flag, every
  // later wait then ends after a few polls, and the item runs to its end on
  // whatever it finds (its request is flagged, its rows are unspecified).
  // A vote on the outcome of each wait measured 1335 -> 1555 us on one prompt
  // of 16384 tokens, one polling lane and a shuffle 1998 us.
  auto wait = [&](uint64_t* bar, int phase) { mbar_wait(bar, phase & 1, &abort_flag); };
  // The next work item of a consumer warp; false at the end (or on a timeout).
  auto take_work = [&](int it, Work& w) -> bool {
    const bool ok = mbar_wait(&w_full[it & 1], (it >> 1) & 1, &abort_flag);
    if (!__all_sync(0xffffffffu, ok && !*(volatile int*)&abort_flag)) return false;
    w = work[it & 1];
    __syncwarp();
    if (lane == 0) mbar_arrive(&w_empty[it & 1]);
    return w.valid;
  };

  // The Q tiles of an item (one warp): row r = (token r / g, head kvh * g + r % g).
  auto load_q = [&](const Work& w) {
    const int tiles = w.nt[1] > 0 ? 2 : 1;
    if (prm.q_tma) {
      if (lane == 0) {
        mbar_expect_tx(&q_full, tiles * L::kTile);
        for (int t = 0; t < tiles; ++t)
#pragma unroll
          for (int h = 0; h < L::DH; ++h)
            tma_load_3d(sbase + t * L::kTile + h * (BM * 128), &tmap_q, h * 64, w.kvh * a.g,
                        w.off + (w.r0 + t * BM) / a.g, &q_full);
      }
      return;
    }
    // by 16-byte asynchronous copies: lane's chunk of every (32 / CPR)-th row,
    // token and head of the row stepped along
    constexpr int CPR = D / 8;        // 16-byte chunks per row
    constexpr int STEP = 32 / CPR;    // rows per round
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q);
    const int ch = lane % CPR, rows = min(tiles * BM, w.n * a.g - w.r0);
    int tok = (w.r0 + lane / CPR) / a.g, head = (w.r0 + lane / CPR) % a.g;
    for (int r = lane / CPR; r < tiles * BM; r += STEP) {
      const int rr = r % BM;
      const uint32_t at = (r / BM) * L::kTile + (ch >> 3) * (BM * 128) + rr * 128 + (((ch & 7) ^ (rr & 7)) << 4);
      if (r < rows)
        cp_async16(sbase + at, q + ((size_t)(w.off + tok) * a.Hq + w.kvh * a.g + head) * D + ch * 8);
      else
        *reinterpret_cast<uint4*>(smem + at) = make_uint4(0, 0, 0, 0);
      for (head += STEP; head >= a.g; head -= a.g) ++tok;
    }
    cp_async_wait();
    fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&q_full);
  };

  // One item's K or V tiles; false after a timeout.  K and V have a producer warp
  // each, so that neither's box issue holds up the other (pages of 16 keys are
  // 16 boxes a tile).  The ring's stages go round in the order of use, K_0, K_1,
  // V_0, K_2, V_1, ..., and each producer takes its own.  Lane i issues the box
  // of page (or 128-row piece) i of a tile; the table is read a tile before.
  auto load_ring = [&](const CUtensorMap* map, const Work& w, int& ld, int is_v) -> bool {
    const int br = prm.box_rows, nb = BN / br, n = max(w.nt[0], w.nt[1]), Lk = w.P + w.n;
    const int32_t* bt = a.block_table + (size_t)w.b * a.max_blocks;
    int bad = 0;
    auto row = [&](int j) { return lane < nb ? box_row(prm, bt, w.kvh, w.k_begin + j * BN + lane * br, Lk, &bad) : 0; };
    int y = row(0);
    for (int j = 0; j < n; ++j) {
      const int y1 = j + 1 < n ? row(j + 1) : 0;
      const int i = ld + (is_v ? (j + 1 < n ? 2 * j + 2 : 2 * n - 1) : (j == 0 ? 0 : 2 * j - 1));
      const int st = i % NST;
      bool go = true;
      if (lane == 0 && i >= NST) go = mbar_wait(&kv_empty[st], (i / NST - 1) & 1, &abort_flag);
      if (!__shfl_sync(0xffffffffu, (int)go, 0)) return false;
      if (lane == 0) {
        mbar_expect_tx(&kv_full[st], L::kTile);
        kv_issued[st] = i;
      }
      __syncwarp();
      if (lane < nb) {
        const uint32_t dst = sbase + L::kOffKV + st * L::kTile + lane * br * 128;
#pragma unroll
        for (int h = 0; h < L::DH; ++h) tma_load_2d(dst + h * (BN * 128), map, h * 64, y, &kv_full[st]);
      }
      y = y1;
    }
    if (!is_v && __any_sync(0xffffffffu, bad) && lane == 0) atomicOr(&a.status[w.b], SPEC_DEV_BAD_BLOCK);
    ld += 2 * n;
    return true;
  };

  // 168 registers a thread hold every role with one 4-byte spill (128 x 152 +
  // 256 x 168 = 62464 of the 384 x 168 launched); a split of 80 and 208 spilled
  // more, in the loading warps
  if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 152;");
  if (warp == 2) {
    // ------------------------------------------------------ work items, Q and V tiles
    // item it + 1 is handed out once item it's loads are out
    if (lane == 0) {
      if (prm.q_tma) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_q)) : "memory");
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_v)) : "memory");
    }
    // item it + 1 is asked for (the launch of a CTA that has not begun is taken
    // over, so that items go to whichever SM is free) while item it runs
    int asked = 0, ld = 0;
    auto ask = [&]() {
      if (lane == 0) {
        mbar_expect_tx(&next_full, 16);
        launch_try_cancel(next_cta, &next_full);
      }
      ++asked;
    };
    auto answer = [&]() -> int {  // the next item, -1 when none is left
      int id = -1;
      if (lane == 0 && mbar_wait(&next_full, (asked - 1) & 1, &abort_flag)) id = launch_cancelled(next_cta);
      if (lane == 0) fence_async_smem();  // read before the next answer is written
      return __shfl_sync(0xffffffffu, id, 0);
    };
    int idx = (int)blockIdx.x;
    for (int it = 0;; ++it) {
      Work w = {};
      if (it > 0) idx = answer();
      while (idx >= 0) {
        ask();
        if (idx == 0) prompt_flag_requests(a, lane, 32);
        w = find_work(prm, order, (uint32_t)idx, lane);
        if (w.valid) break;
        idx = answer();
      }
      bool ok = true;
      if (it >= 2 && lane == 0) ok = mbar_wait(&w_empty[it & 1], ((it >> 1) - 1) & 1, &abort_flag);
      if (!__shfl_sync(0xffffffffu, ok, 0)) break;
      if (lane == 0) {
        work[it & 1] = w;
        mbar_arrive(&w_full[it & 1]);
      }
      if (!w.valid) break;
      if (lane == 0 && it >= 1) ok = mbar_wait(&q_empty, (it - 1) & 1, &abort_flag);
      if (!__shfl_sync(0xffffffffu, ok, 0)) break;
      load_q(w);
      if (lane == 0) q_issued = it;
      if (!load_ring(&tmap_v, w, ld, 1)) break;
    }
    if (lane == 0 && asked > 0) mbar_drain(&next_full, (asked - 1) & 1);
  } else if (warp == 0) {
    // ------------------------------------------------------ K producer
    if (lane == 0) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_k)) : "memory");
    Work w;
    int ld = 0;
    for (int it = 0; take_work(it, w); ++it)
      if (!load_ring(&tmap_k, w, ld, 0)) break;
  } else if (warp == 1 || warp == 3) {
    // ------------------------------------------------------ MMA issuers
    // warp 1: tile 0, warp 3: tile 1.  The whole warp runs the loop (so that
    // descriptors stay warp-uniform) and one elected lane issues.  A tile that
    // has no work in a step still gives the step's stages back.
    const int t = warp >> 1;
    constexpr uint32_t idesc_qk = idesc_bf16(BN, 0), idesc_pv = idesc_bf16(D, 1);
    const uint64_t qd = smem_desc_sw128(sbase + t * L::kTile, 16, 1024);
    const uint64_t kdesc = smem_desc_sw128(sbase + L::kOffKV, 16, 1024);
    const uint64_t vdesc = smem_desc_sw128(sbase + L::kOffKV, BN * 128, 1024);
    const uint32_t tS = tmem + t * BN, tO = tmem + 2 * BN + t * 128;
    const bool leader = elect_one();
    int ld = 0, cs = 0, turns = 0;  // loads and score tiles used, turns taken
    // the elected lane's issues
    auto qk = [&](int i) {
      const uint64_t kd = kdesc + (uint64_t)((i % NST) * (L::kTile >> 4));
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t o = ((kk >> 2) * (BM * 128) + (kk & 3) * 32) >> 4;
        umma_bf16(tS, qd + o, kd + o, idesc_qk, kk > 0 ? 1u : 0u);
      }
      umma_commit(&s_full[t]);
    };
    auto pv = [&](int h, uint64_t vd, bool first) {
#pragma unroll
      for (int kk = 0; kk < HC / 16; ++kk)
        umma_bf16_ts(tO, tS + h * (HC / 2) + kk * 8, vd + (uint64_t)(((h * (HC / 16) + kk) * 2048) >> 4), idesc_pv,
                     first && kk == 0 ? 0u : 1u);
      umma_commit(&o_done[t][h]);
    };
    Work w;
    for (int it = 0; take_work(it, w); ++it) {
      const int nt = t == 0 ? w.nt[0] : w.nt[1], n = max(w.nt[0], w.nt[1]);
      // load numbers: K_0 = 0, K_j = 2j - 1, V_j = 2j + 2 (the last V: 2n - 1)
      wait(&q_full, it);
      wait(&kv_full[ld % NST], ld / NST);
      tc_fence_after();
      if (leader) {
        if (nt > 0) qk(ld);
        umma_commit(&kv_empty[ld % NST]);
        if (n == 1) umma_commit(&q_empty);
      }
      for (int j = 0; j < n; ++j) {
        const int iv = ld + (j + 1 < n ? 2 * j + 2 : 2 * n - 1), ik = ld + 2 * j + 1;
        const uint64_t vd = vdesc + (uint64_t)((iv % NST) * (L::kTile >> 4));
        wait(&kv_full[iv % NST], iv / NST);
        if (j + 1 < n) wait(&kv_full[ik % NST], ik / NST);
        if (t == 1 || turns > 0) wait(&turn[t], t == 1 ? turns : turns - 1);
        ++turns;
        if (j < nt) {
          wait(&p_full[t][0], cs);
          tc_fence_after();
          if (leader) pv(0, vd, j == 0);
          wait(&p_full[t][1], cs);
          ++cs;
          tc_fence_after();
        }
        // short branches: one long branch of the elected lane for PV, QK and
        // the commits measured 1320 -> 1490 us on one prompt of 16384 tokens
        if (j < nt && leader) pv(1, vd, false);
        if (j + 1 < nt) {
          tc_fence_after();
          if (leader) {
            qk(ik);
            mbar_arrive(&turn[t ^ 1]);
          }
        } else if (leader) {
          mbar_arrive(&turn[t ^ 1]);
        }
        if (leader) {
          umma_commit(&kv_empty[iv % NST]);
          if (j + 1 < n) umma_commit(&kv_empty[ik % NST]);
          if (j + 2 == n) umma_commit(&q_empty);  // the item's last QK is out
        }
      }
      ld += 2 * n;
    }
    if (leader) {  // every MMA has completed before TMEM is freed
      umma_commit(&drain[t]);
      mbar_drain(&drain[t], 0);
    }
  } else {
    // ------------------------------------------------------ softmax, epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
    const int t = (warp - 4) >> 2, quad = warp & 3;
    const int r = quad * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const uint32_t tS = tmem + t * BN + lane_off, tO = tmem + 2 * BN + t * 128 + lane_off;
    const float c2 = a.scale_log2;
    const float2 c22 = make_float2(c2, c2);
    int ld = 0, cs = 0;  // loads so far (as the MMA warp counts them), score tiles of this row tile
    float m = 0.0f, l = 0.0f;  // the row's reference (log2 domain) and sum
    float limit = kSumLimit;
    // weights 2^(x c - ref) of 32 columns, `vis` of them visible, packed to bf16
    // in pk[0 .. 15] (each off by at most half a bf16 step); returns the fp32 sum
    // of the packed ones: numerator and denominator hold the same weights, so that
    // a key that stands alone gives its V.  Summing the weights before they are
    // rounded takes fewer instructions (one prompt of 16384: 1258 us against 1320).
    auto weights = [&](uint32_t (&x)[32], int vis, float ref, uint32_t* pk) -> float {
      if (!__all_sync(0xffffffffu, vis >= 32)) {
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (e >= vis) x[e] = 0xff800000u;
      }
      const float2 neg = make_float2(-ref, -ref);
      float2 acc0 = make_float2(0.0f, 0.0f), acc1 = acc0;
#pragma unroll
      for (int e = 0; e < 32; e += 2) {
        const float2 z = __ffma2_rn(make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), c22, neg);
        const float2 p = make_float2(fast_exp2(z.x), fast_exp2(z.y));
        const __nv_bfloat162 h2 = __floats2bfloat162_rn(p.x, p.y);
        const uint32_t u = *reinterpret_cast<const uint32_t*>(&h2);
        pk[e >> 1] = u;
        if (e & 2) add_bf16x2(acc1, u);
        else add_bf16x2(acc0, u);
      }
      return (acc0.x + acc0.y) + (acc1.x + acc1.y);
    };
    // Whether half weights that sum to `sum` need another reference (a NaN stays
    // one against any).
    auto unfit = [&](float sum, int vis) -> bool {
      return __any_sync(0xffffffffu, sum >= limit || (l == 0.0f && vis > 0 && sum < 1.0f / kSumLimit));
    };
    // Half h again, from its scores in tensor memory, against a reference that
    // covers it.  A row with nothing summed yet takes its maximum; a row with a
    // sum takes it where it is larger, and scales the sum and O.
    auto redo = [&](int h, int vis, bool have_o, uint32_t (&pk)[HC / 2], float& sum) {
      uint32_t x[32];
      float mx = -INFINITY;
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        tmem_ld32(tS + h * HC + c * 32, x);
        tmem_wait_ld(x);
#pragma unroll
        for (int e = 0; e < 32; ++e) mx = fmaxf(mx, c * 32 + e < vis ? __uint_as_float(x[e]) : -INFINITY);
      }
      float f = 1.0f;
      if (l == 0.0f) {
        if (mx != -INFINITY) m = mx * c2;  // O holds zeros
      } else if (mx * c2 > m) {
        f = fast_exp2(m - mx * c2);
        l *= f;
        m = mx * c2;
      }
      sum = 0.0f;
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        tmem_ld32(tS + h * HC + c * 32, x);
        tmem_wait_ld(x);
        sum += c == 0 ? weights(x, vis, m, pk) : weights(x, vis - 32, m, pk + 16);
      }
      if (!have_o || !__any_sync(0xffffffffu, f != 1.0f)) return;
      // O holds every earlier half once the last of them has completed: this
      // tile's first, or the previous tile's second (one barrier for each, so
      // that a wait is never two phases behind)
      wait(&o_done[t][h ^ 1], h == 1 ? cs : cs - 1);
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        tmem_ld32(tO + c * 32, x);
        tmem_wait_ld(x);
#pragma unroll
        for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * f);
        tmem_st32(tO + c * 32, x);
      }
    };
    Work w;
    for (int it = 0; take_work(it, w); ++it) {
      const int nt = t == 0 ? w.nt[0] : w.nt[1], n = max(w.nt[0], w.nt[1]), Lk = w.P + w.n;
      const int row = w.r0 + t * BM + r;
      const bool valid = row < w.n * a.g;
      const int tok = valid ? row / a.g : w.n - 1;
      const int lim = w.P + tok + 1 - w.k_begin;  // visible keys of this range
      // rows behind the request (the next one's q, or NaN) have no say in a redo
      limit = valid ? kSumLimit : NAN;
      m = 0.0f;
      l = valid ? 0.0f : 1.0f;
      for (int j = 0; j < nt; ++j, ++cs) {
        wait(&s_full[t], cs);
        tc_fence_after();
        const int k0 = w.k_begin + j * BN;
        if (k0 + BN > Lk) {
          // the tile reaches past the request: its V rows there are zeroed, so
          // that no stale bits (NaN among them) meet a zero probability
          const int iv = ld + 2 * n - 1;  // only the range's last tile can
          wait(&kv_full[iv % NST], iv / NST);
          const int zr = Lk - k0;
          uint8_t* vst = smem + L::kOffKV + (iv % NST) * L::kTile;
          for (int i = r; i < (BN - zr) * L::DH * 8; i += BM) {
            const int rr = zr + i / (L::DH * 8), rest = i % (L::DH * 8);
            *reinterpret_cast<uint4*>(vst + (rest >> 3) * (BN * 128) + rr * 128 + ((rest & 7) << 4)) =
                make_uint4(0, 0, 0, 0);
          }
          fence_async_smem();
        }
        // quarters of 32 columns, each loaded beside the weights of the one
        // before; P of a half goes back once its weights are known to fit.  The
        // loop stays rolled: short items run each part of the code once, and
        // what they wait for is instructions (64 prompts of 512 tokens: 224 us
        // with the halves unrolled, 199 rolled, 257 with the output's chunks
        // unrolled as well).
        const int vis = lim - j * BN;  // visible columns of this tile
        uint32_t x[32], y[32], pk[HC / 2];
        tmem_ld32(tS, x);
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          tmem_wait_ld(x);
          tmem_ld32(tS + h * HC + 32, y);
          float sum = weights(x, vis - h * HC, m, pk);
          tmem_wait_ld(y);
          if (h == 0) tmem_ld32(tS + HC, x);
          sum += weights(y, vis - h * HC - 32, m, pk + 16);
          if (unfit(sum, vis - h * HC)) redo(h, vis - h * HC, j > 0 || h > 0, pk, sum);
          l += sum;
          tmem_st32(tS + h * (HC / 2), pk);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[t][h]);
        }
      }
      ld += 2 * n;
      if (nt == 0) continue;
      // epilogue: this thread's row
      wait(&o_done[t][1], cs - 1);
      tc_fence_after();
      const size_t orow = (size_t)(w.off + tok) * a.Hq + w.kvh * a.g + (valid ? row % a.g : 0);
      const float inv = 1.0f / l;
      // 64 bytes of every row of the warp, one 16-byte piece u[i] after another
      // in each thread: four lanes trade pieces so that each store writes 64
      // contiguous bytes of 8 rows (16 bytes of 32 rows cost four times the
      // address passes).
      uint32_t rows4[4];  // output rows of the four lanes, 0xffffffff: not written
#pragma unroll
      for (int s = 0; s < 4; ++s)
        rows4[s] = __shfl_sync(0xffffffffu, valid ? (uint32_t)orow : 0xffffffffu, (lane & 28) + s);
      auto store_rows = [&](char* base, int row_bytes, uint4 (&u)[4]) {
        transpose4(u, lane);
#pragma unroll
        for (int s = 0; s < 4; ++s)
          if (rows4[s] != 0xffffffffu)
            *reinterpret_cast<uint4*>(base + (size_t)rows4[s] * row_bytes + (lane & 3) * 16) = u[s];
      };
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        tmem_ld32(tO + c * 32, o);
        tmem_wait_ld(o);
        if (a.splits == 1) {
          uint4 u[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              __nv_bfloat162 h2 = __floats2bfloat162_rn(__uint_as_float(o[8 * i + 2 * e]) * inv,
                                                        __uint_as_float(o[8 * i + 2 * e + 1]) * inv);
              p[e] = *reinterpret_cast<uint32_t*>(&h2);
            }
            u[i] = make_uint4(p[0], p[1], p[2], p[3]);
          }
          store_rows(static_cast<char*>(a.out) + c * 64, 2 * D, u);
        } else {
          char* ws = reinterpret_cast<char*>(a.ws_o + (size_t)w.split * a.T * a.Hq * D);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint4 u[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int at = 16 * i + 4 * e;
              u[e] = make_uint4(o[at], o[at + 1], o[at + 2], o[at + 3]);
            }
            store_rows(ws + c * 128 + i * 64, 4 * D, u);
          }
        }
      }
      if (valid && a.splits > 1)
        *reinterpret_cast<float2*>(a.ws_ml + ((size_t)w.split * a.T * a.Hq + orow) * 2) = make_float2(l > 0.0f ? m : -INFINITY, l);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (abort_flag) {
    // every copy has landed before the CTA exits (without a timeout the MMA
    // warps have waited for each); which of the CTA's items were lost is not
    // kept: every request is flagged
    if (threadIdx.x == 0) {
      for (int st = 0; st < NST; ++st)
        if (kv_issued[st] >= 0) mbar_drain(&kv_full[st], (kv_issued[st] / NST) & 1);
      if (q_issued >= 0) mbar_drain(&q_full, q_issued & 1);
    }
    for (int b = threadIdx.x; b < a.B; b += kThreads) atomicOr(&a.status[b], SPEC_DEV_TIMEOUT);
  }
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

}  // namespace ptc

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
typedef CUresult (*PromptEncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static PromptEncodeFn prompt_encode_fn() {
  static const PromptEncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PromptEncodeFn>(p);
  }();
  return fn;
}

static bool prompt_map(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                       const cuuint32_t* box) {
  const PromptEncodeFn enc = prompt_encode_fn();
  const cuuint32_t one[3] = {1, 1, 1};
  return enc && enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box, one,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
static cudaError_t launch_d(const PromptArgs& a, const PromptPlan& p, cudaStream_t stream) {
  ptc::Params prm;
  prm.a = a;
  prm.box_rows = std::min(a.block_size, ptc::BN);
  prm.bs_log2 = 0;
  while ((1 << prm.bs_log2) < a.block_size) ++prm.bs_log2;
  prm.rows_total = (long long)a.num_blocks * a.Hkv * a.block_size;
  const long long items = p.tiles * a.Hkv * p.splits;
  alignas(64) CUtensorMap mk, mv, mq;
  {
    const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)prm.rows_total}, strides[1] = {(cuuint64_t)D * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)prm.box_rows};
    if (!prompt_map(&mk, a.k_cache, 2, dims, strides, box) || !prompt_map(&mv, a.v_cache, 2, dims, strides, box))
      return cudaErrorInvalidValue;
  }
  // Q [T][Hq][D] as (columns, heads, tokens): a (64, g, 128 / g) box is one
  // 64-column half of a row tile
  prm.q_tma = ptc::BM % a.g == 0;
  if (prm.q_tma) {
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)a.Hq, (cuuint64_t)a.T};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)a.Hq * D * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)a.g, (cuuint32_t)(ptc::BM / a.g)};
    if (!prompt_map(&mq, a.q, 3, dims, strides, box)) return cudaErrorInvalidValue;
  } else {
    mq = mk;  // not read
  }
  const int dyn = (int)ptc::Layout<D>::kDyn;
  const cudaError_t e = cudaFuncSetAttribute(ptc::prompt_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, dyn);
  if (e != cudaSuccess) return e;
  // one CTA per item; the CTAs that run take over the launches of the others
  ptc::prompt_tc_kernel<D><<<(unsigned)items, ptc::kThreads, dyn, stream>>>(mk, mv, mq, prm);
  return cudaGetLastError();
}

cudaError_t launch_prompt_tc(const PromptArgs& a, const PromptPlan& p, cudaStream_t stream) {
  return a.D == 64 ? launch_d<64>(a, p, stream) : launch_d<128>(a, p, stream);
}

}  // namespace spectree
