// Log probabilities of given tokens, with the entropy of their distribution,
// the token's rank and the top alternatives.
//
// For one row of logits x, inverse temperature tau and given token t, with
// any reference r and d_i = x_i - r:
//   S = sum_i e^(tau d_i),  W = sum_i e^(tau d_i) d_i
//   log p(t) = tau d_t - log S
//   H = -sum_i p_i log p_i = log S - tau W / S
//   rank(t) = number of tokens ranked before t (larger logit, equal logits by
//             lower id, NaN last)
// Every value comes from one read of the row: each thread keeps (r, S, W)
// with r the largest logit it has seen, moves to a larger r once per batch of
// 16 entries, and the partials merge by the same rule across the warp, the CTA
// and the row's cluster, always in the same order.
//
// The row is the only traffic that counts.  A producer warp brings it by bulk
// copies through a shared-memory ring, so that what is in flight (three CTAs an
// SM, 64 KB each) does not hang on registers, and runs ahead into the CTA's next
// row while this one is summed up.  Measured on 2048 rows of 128256 fp32 logits,
// 30 % of the tokens unlikely ones: 181 us with k = 0 (5.8 TB/s), 235 us with
// k = 20; loads into registers ahead of each batch: 250 us with k = 0.  What
// bounds it: with k = 0 the memory (half of a stage's 2400 cycles are spent
// waiting for it); with k = 20 a warp's chain through a batch, some 1100 cycles
// and the alternatives' on top, at half of the issue slots (bf16 logits take as
// long as fp32 ones).  2048 rows are five rounds of 456 CTAs; the rest of the last
// round, a row to two CTAs, took 8 us less on 500 rows and 14 us more on 2048.
// The rank looks at a lane's entries only when their maximum reaches the given
// token's logit, and the alternatives only when it reaches the CTA's bar (below).
// A bar per warp let eight times as many entries through (314 us), and with the
// insertion inlined per entry the whole took 924 us.  Eight consumer warps in
// three CTAs of 72 registers; four in five CTAs measured 353 us.
//
// One cluster of C CTAs per row: the most that leave the call within 8 / 3 CTAs
// an SM (three fit, but clusters do not fill every SM; one that waits for room
// doubles the call), with at least 2048 entries each.  V 128256, k = 20, by C =
// 1, 2, 4, 8: 16 rows 46, 35, 27, 23 us; 100 rows 50, 39, 37, 50; 200 rows 54,
// 46, 60, 111; 250 rows 56, 70, 91, 144.
#include <algorithm>
#include <climits>

#include <cooperative_groups.h>

#include "tcgen05.cuh"
#include "topk.cuh"

namespace cg = cooperative_groups;

namespace spectree {

constexpr int kLpWarps = 8;                          // consumer warps (cta_bar compares 8 scores)
constexpr int kLpThreads = kLpWarps * 32 + 32;       // and the producer warp
constexpr int kLpBatch = 16;                         // entries per lane and stage
constexpr int kLpEntries = kLpWarps * 32 * kLpBatch; // entries per stage: 16 KB of fp32, 8 KB of bf16
constexpr int kLpDyn = 64 * 1024;                    // the ring: 4 stages of fp32, 8 of bf16; three CTAs an SM
constexpr int kLpMaxCluster = 8;
constexpr int kLpMaxLive = 1024;  // requests whose accepted lengths a CTA sums up for itself

__device__ __forceinline__ float lp_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// max that keeps NaN (fmaxf drops it)
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// max(a, b, c) that keeps NaN
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float y;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

// S and W against the reference r; r = -inf: nothing above -inf seen yet.  A
// NaN stays NaN through every merge.  c = tau log2 e.
struct SoftStats {
  float r = -INFINITY, s = 0.0f, w = 0.0f;

  // the same sums against a larger reference
  __device__ __forceinline__ void raise(float to, float c) {
    if (r == to) return;
    if (r == -INFINITY) {
      s = w = 0.0f;
    } else {
      const float d = r - to;  // <= 0; -inf when `to` is +inf
      const float f = lp_exp2(d * c);
      // f > 0 leaves |d| below 88 / tau, so that s d is finite; a NaN has f NaN
      w = f == 0.0f ? 0.0f : f * fmaf(s, d, w);
      s *= f;
    }
    r = to;
  }
  // the statistics of N neighbouring lanes together: their largest reference,
  // one rescaling, plain sums
  template <int N> __device__ __forceinline__ void reduce(float c) {
    float to = r;
#pragma unroll
    for (int o = N / 2; o; o >>= 1) to = max_nan(to, __shfl_xor_sync(0xffffffffu, to, o));
    raise(to, c);
#pragma unroll
    for (int o = N / 2; o; o >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, o);
      w += __shfl_xor_sync(0xffffffffu, w, o);
    }
  }
  __device__ __forceinline__ void merge(SoftStats o, float c) {
    const float to = max_nan(r, o.r);
    raise(to, c);
    o.raise(to, c);
    s += o.s;
    w += o.w;
  }
};

// One entry per work item: a row of the logits and the token given for it.
struct LpArgs {
  const void* logits;
  const int32_t* tokens;      // [T], or emitted [B][n_max]
  const int32_t* off;         // [B + 1]
  const int32_t* path;        // [B][n_max] or NULL (packed rows)
  const int32_t* accept_len;  // [B] with path
  const float* inv_temp;      // [B] or NULL
  float *logprob, *entropy, *top_logprobs;
  int32_t *rank, *top_tokens, *status;
  int B, T, n_max, V, k, C;
  int live;  // path call: clusters go round the accepted entries alone
};

template <typename T> __device__ __forceinline__ void lp_unpack(uint4 v, float (&x)[16 / sizeof(T)]);
template <> __device__ __forceinline__ void lp_unpack<float>(uint4 v, float (&x)[4]) {
  x[0] = __uint_as_float(v.x);
  x[1] = __uint_as_float(v.y);
  x[2] = __uint_as_float(v.z);
  x[3] = __uint_as_float(v.w);
}
template <> __device__ __forceinline__ void lp_unpack<__nv_bfloat16>(uint4 v, float (&x)[8]) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}

// A float's order as a signed integer (both ways the same mapping).
__device__ __forceinline__ int float_order(float v) {
  const int i = __float_as_int(v);
  return i >= 0 ? i : i ^ 0x7fffffff;
}
__device__ __forceinline__ float order_float(int i) { return __int_as_float(i >= 0 ? i : i ^ 0x7fffffff); }

// Barrier of the consumer warps.
__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kLpWarps * 32) : "memory"); }

// The next float below (finite and infinite alike; -inf stays).
__device__ __forceinline__ float before_float(float v) {
  return v == -INFINITY ? v : order_float(float_order(v == 0.0f ? -0.0f : v) - 1);
}

__device__ __forceinline__ void write_none(const LpArgs& a, long long entry, int thread) {
  if (thread == 0) {
    a.logprob[entry] = NAN;
    if (a.entropy) a.entropy[entry] = NAN;
    if (a.rank) a.rank[entry] = -1;
  }
  if (thread < a.k) {
    if (a.top_tokens) a.top_tokens[entry * a.k + thread] = -1;
    if (a.top_logprobs) a.top_logprobs[entry * a.k + thread] = NAN;
  }
}

// Rows are read once: their lines are the first to leave L2 (2048 rows of 128256
// fp32, k = 0: 190 -> 181 us; k = 20: 238 -> 233; rows of 1000: 80 -> 82).
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  uint64_t once;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(once));
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
          tc5::smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(tc5::smem_u32(bar)), "l"(once)
      : "memory");
}

template <typename T>
__global__ void __launch_bounds__(kLpThreads, 3) logprobs_kernel(const LpArgs a, long long entries) {
  constexpr int VEC = 16 / sizeof(T);
  constexpr int NE = kLpBatch, NV = NE / VEC;     // entries and vectors per lane and stage
  constexpr int kLpChunk = kLpEntries / VEC;      // vectors per stage
  constexpr int kLpStages = kLpDyn / (kLpChunk * 16);
  extern __shared__ __align__(128) uint4 ring[];
  __shared__ unsigned long long s_keys[kLpWarps * 32];  // the warps' keys that reach the last bar
  __shared__ unsigned long long cres[kLpMaxCluster][32];  // leader: the CTAs' lists
  __shared__ SoftStats wst[kLpWarps], cst[kLpMaxCluster];
  __shared__ int wbef[kLpWarps], cbef[kLpMaxCluster];
  __shared__ int s_mth[kLpWarps];     // each warp's m-th best score, in float_order
  __shared__ int s_n;
  __shared__ int s_live[kLpMaxLive];  // accepted entries before each request
  __shared__ int s_total, abort_flag, s_last[kLpStages];  // s_last: the last copy into each stage
  __shared__ uint64_t full[kLpStages], empty[kLpStages];
  cg::cluster_group cluster = cg::this_cluster();
  const int C = a.C, part = (int)cluster.block_rank();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long first = blockIdx.x / C, step = gridDim.x / C;
  const int k = a.k;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kLpStages; ++i) {
      tc5::mbar_init(&full[i], 1);
      tc5::mbar_init(&empty[i], kLpWarps);
      s_last[i] = -1;
    }
    abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (a.live && warp == 0) {
    // the accepted entries alone are gone through, numbered request by request
    int at = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      const int b = b0 + lane;
      const int n_acc = b < a.B ? a.accept_len[b] : 0;
      if (n_acc > a.n_max && blockIdx.x == 0) atomicOr(&a.status[b], SPEC_DEV_BAD_PATH);
      const int n = n_acc > 0 && n_acc <= a.n_max ? n_acc : 0;
      int incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      if (b < a.B) s_live[b] = at + incl - n;
      at += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) s_total = at;
  }
  if (C > 1) cluster.sync();  // its CTAs run: partials may be written to the leader's shared memory
  else __syncthreads();
  if (a.live) {
    for (long long e = blockIdx.x * kLpWarps + warp; warp < kLpWarps && e < entries; e += (long long)gridDim.x * kLpWarps) {
      const int n = a.accept_len[(int)(e / a.n_max)];
      if ((int)(e % a.n_max) >= n || n > a.n_max) write_none(a, e, lane);
    }
    entries = s_total;
  }

  int chunks = 0;  // stages used so far
  for (long long item = first; item < entries; item += step) {
    // ---- the item's entry, row and token
    long long entry = item, row = item;
    int b = 0, token = -1, bad = 0;
    bool none = false;  // nothing to compute: the outputs say so
    if (a.path) {
      if (a.live) {
        int lo = 0, hi = a.B;  // the last request with s_live[lo] <= item
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (s_live[mid] <= item) lo = mid;
          else hi = mid;
        }
        b = lo;
        entry = (long long)b * a.n_max + (item - s_live[b]);
      } else {
        b = (int)(entry / a.n_max);
        const int n_acc = a.accept_len[b];
        none = (int)(entry % a.n_max) >= n_acc || n_acc > a.n_max;
        if (n_acc > a.n_max) bad = SPEC_DEV_BAD_PATH;
      }
      if (!none) {
        const int off = a.off[b], n = a.off[b + 1] - off, p = a.path[entry];
        token = a.tokens[entry];
        if (off < 0 || n < 0 || n > a.T - off || p < 0 || p >= n) bad |= SPEC_DEV_BAD_PATH;
        row = (long long)off + p;
      }
    } else if (warp < kLpWarps) {  // the producer needs the row alone
      int lo = 0, hi = a.B;        // the last request with off[lo] <= entry
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.off[mid] <= entry) lo = mid;
        else hi = mid;
      }
      b = lo;
      token = a.tokens[entry];
      none = entry < a.off[b] || entry >= a.off[b + 1];  // a row no request owns
    }
    // a path entry without a row is left out by every warp of the cluster; a
    // row that is read for nothing is settled at the end
    const bool skip = a.path && (none || bad);

    // ---- the row: a head up to the first 16-byte boundary, 16-byte vectors, a tail
    const T* src = static_cast<const T*>(a.logits) + row * a.V;
    const int mis = (int)((reinterpret_cast<uintptr_t>(src) & 15) / sizeof(T));
    const int head = min(a.V, mis ? VEC - mis : 0);
    const int nvec = (a.V - head) / VEC;
    const int tail0 = head + nvec * VEC;
    const int per = (nvec + C - 1) / C;
    const int v0 = min(nvec, part * per), v1 = min(nvec, v0 + per);
    const int n_chunks = skip ? 0 : (v1 - v0 + kLpChunk - 1) / kLpChunk;
    if (warp == kLpWarps) {  // ---- producer
      if (lane == 0) {
        for (int i = 0; i < n_chunks; ++i) {
          const int u = chunks + i, st = u % kLpStages;
          if (u >= kLpStages && !tc5::mbar_wait(&empty[st], (u / kLpStages - 1) & 1, &abort_flag)) break;
          const uint32_t bytes = 16u * (uint32_t)min(kLpChunk, v1 - v0 - i * kLpChunk);
          tc5::mbar_expect_tx(&full[st], bytes);
          s_last[st] = u;
          bulk_load(ring + st * kLpChunk, reinterpret_cast<const uint4*>(src + head) + v0 + i * kLpChunk, bytes, &full[st]);
        }
      }
      chunks += n_chunks;
      if (C > 1) {  // a cluster's barriers take every warp; alone, the producer runs ahead into the next rows
        if (!skip) cluster.sync();
        if (item + step < entries) cluster.sync();
      }
      continue;
    }
    float tau = 1.0f;
    if (a.inv_temp && !none) {
      tau = a.inv_temp[b];
      if (!(tau >= 1e-30f && tau < INFINITY)) bad |= SPEC_DEV_BAD_TEMP;
    }
    if (!none && (token < (a.path ? 0 : -1) || token >= a.V)) {
      bad |= SPEC_DEV_BAD_TOKEN;
      token = -1;
    }
    if (!skip) {
      const float c = fminf(tau * 1.4426950408889634f, 3.4e38f);  // finite: 0 times it is 0
      const float2 cc = make_float2(c, c);
      const float xt = token >= 0 ? to_f32(src[token]) : INFINITY;  // no token: no entry is above it
      SoftStats st;
      WarpTop top;
      int before = 0;
      // The bar: the w-th largest of the warps' m-th best scores, w m >= k, is
      // reached by k entries of the CTA, and no entry below it is among the k
      // best.  w of about five eighths of the nw warps that work on this row.
      const int nw = n_chunks > 0 ? min(kLpWarps, (v1 - v0 + NV * 32 - 1) / (NV * 32)) : 1;
      const int most = (5 * nw + 7) / 8, m = (k + most - 1) / most, w = m > 0 ? (k + m - 1) / m : 0;
      float mth = -INFINITY;
      if (threadIdx.x < kLpWarps) s_mth[threadIdx.x] = float_order(-INFINITY);
      if (threadIdx.x == 0) s_n = 0;
      consumers_sync();
      auto cta_bar = [&]() -> float {
        // lane 8 j + i: is score j, or j + 4, above score i; lane i then counts.
        // The other warps raise their scores meanwhile: each is read once (read
        // again, a score could be above its own earlier value, which then looked
        // like one rank more and left the bar too high).
        const int v = *(const volatile int*)&s_mth[lane & 7];
        const int mine = __shfl_sync(0xffffffffu, v, lane & 7);
        const int lo = __shfl_sync(0xffffffffu, v, lane >> 3), hi = __shfl_sync(0xffffffffu, v, (lane >> 3) + 4);
        const unsigned col = 0x01010101u << (lane & 7);
        const int above = __popc(__ballot_sync(0xffffffffu, lo > mine) & col) + __popc(__ballot_sync(0xffffffffu, hi > mine) & col);
        return order_float(__reduce_min_sync(0xffffffffu, above < w ? mine : INT_MAX));
      };
      // A batch of entries, one lane's x[0 .. N - 1]; those that are not there
      // hold -inf.  The sums:
      auto sums = [&](auto& x, float mx) {
        constexpr int N = sizeof(x) / sizeof(float);
        // entries of -inf weigh nothing; the reference stays, since one of NaN would
        // be lost to -inf (nothing seen yet), and the row's NaN with it
        if (mx == -INFINITY) return;
        if (!(mx <= st.r)) st.raise(mx, c);
        float s = 0.0f, w = NAN;
        if constexpr (N > 1) {
          const float2 neg = make_float2(-st.r, -st.r);
          float2 s2 = make_float2(0.0f, 0.0f), w2 = s2;
#pragma unroll
          for (int q = 0; q < N; q += 2) {
            const float2 d = __fadd2_rn(make_float2(x[q], x[q + 1]), neg);
            const float2 z = __fmul2_rn(d, cc);
            const float2 e = make_float2(lp_exp2(z.x), lp_exp2(z.y));
            s2 = __fadd2_rn(s2, e);
            w2 = __ffma2_rn(e, d, w2);
          }
          s = s2.x + s2.y;
          w = w2.x + w2.y;
        }
        if (w != w) {
          // a weight of 0 at an infinite distance (or a NaN, which stays): again,
          // with the distance held finite
          s = w = 0.0f;
#pragma unroll
          for (int q = 0; q < N; ++q) {
            const float d = max_nan(x[q] - st.r, -3e38f), e = lp_exp2(d * c);
            s += e;
            w = fmaf(e, d, w);
          }
        }
        st.s += s;
        st.w += w;
      };
      // The given token's rank: entry q has id `id(q)` and is there if in(q).
      auto count = [&](auto& x, auto id, auto in) {
        constexpr int N = sizeof(x) / sizeof(float);
#pragma unroll
        for (int q = 0; q < N; ++q) {
          const bool equal = x[q] == xt || (x[q] != x[q] && xt != xt);
          before += in(q) && (x[q] > xt || (xt != xt && x[q] == x[q]) || (equal && id(q) < token));
        }
      };
      // The alternatives, when a lane's maximum reaches the bar (as last seen, then
      // as it is now): `offer` takes the lanes that do.
      auto pick = [&](float mx, auto offer) {
        if (!__any_sync(0xffffffffu, !(mx < top.bar))) return;
        top.floor = fmaxf(top.floor, cta_bar());
        top.bar = fmaxf(top.bar, top.floor);
        const unsigned reach = __ballot_sync(0xffffffffu, !(mx < top.bar));
        if (!reach) return;
        offer(reach);
        if (m > 0) {
          const float now = key_score(__shfl_sync(0xffffffffu, top.list, m - 1));
          if (now > mth) {
            mth = now;
            if (lane == 0) *(volatile int*)&s_mth[warp] = float_order(now);
          }
        }
      };
      for (int i = 0; i < n_chunks; ++i) {
        const int u = chunks + i, sg = u % kLpStages;
        const int n = min(kLpChunk, v1 - v0 - i * kLpChunk);       // vectors of the stage
        const int x0 = head + (v0 + i * kLpChunk) * VEC;           // its first entry
        const uint4* sv = ring + sg * kLpChunk;
        const int j0 = warp * NV * 32 + lane;
        tc5::mbar_wait(&full[sg], (u / kLpStages) & 1, &abort_flag);
        float x[NE], mx = -INFINITY;
        const bool here = warp * NV * 32 < n;
        auto id = [&](int q) { return x0 + (j0 + (q / VEC) * 32) * VEC + q % VEC; };
        auto in = [&](int q) { return j0 + (q / VEC) * 32 < n; };
        if (here) {
#pragma unroll
          for (int q = 0; q < NV; ++q) lp_unpack<T>(sv[j0 + q * 32], *reinterpret_cast<float(*)[VEC]>(x + q * VEC));
          if (n < kLpChunk) {  // past the end: an earlier stage's values, or none
#pragma unroll
            for (int q = 0; q < NE; ++q) x[q] = in(q) ? x[q] : -INFINITY;
          }
          mx = x[0];
#pragma unroll
          for (int q = 1; q + 1 < NE; q += 2) mx = max3_nan(mx, x[q], x[q + 1]);
          mx = max_nan(mx, x[NE - 1]);
          sums(x, mx);
          if (!(mx < xt)) {
            const bool lower = x0 + n * VEC <= token, higher = x0 > token;  // every id of the stage
            if (n == kLpChunk && (lower || higher) && xt > -INFINITY) {
              // equal logits of lower ids count too; an entry is above the bar where
              // bar - x has its sign set (+0 for equal ones, NaN positive)
              const float bar = lower ? before_float(xt) : xt + 0.0f;
              unsigned signs = 0;
#pragma unroll
              for (int q = 0; q < NE; q += 2) {
                const float2 d = __ffma2_rn(make_float2(x[q], x[q + 1]), make_float2(-1.0f, -1.0f), make_float2(bar, bar));
                signs = __funnelshift_l(__float_as_uint(d.x), signs, 1);
                signs = __funnelshift_l(__float_as_uint(d.y), signs, 1);
              }
              before += __popc(signs);
            } else {
              count(x, id, in);
            }
          }
        }
        if (k > 0) {
          if (i == 0) {
            // before any list is filled, from the lanes' maxima
            mth = WarpTop::nth_largest(mx, m - 1, lane);
            if (here && lane == 0) *(volatile int*)&s_mth[warp] = float_order(mth);
            consumers_sync();
          }
          if (here)
            pick(mx, [&](unsigned reach) {
              const T* se = reinterpret_cast<const T*>(sv);
              if (__popc(reach) > 6) {  // a row's beginning: an entry of each lane a round
                uint32_t hits = 0;
                if (!(mx < top.bar)) {
#pragma unroll
                  for (int q = 0; q < NE; ++q) hits |= !(x[q] < top.bar) ? 1u << q : 0u;
                }
#pragma unroll 1
                while (__any_sync(0xffffffffu, hits)) {
                  const int q = __ffs(hits) - 1, at = (j0 + (q / VEC) * 32) * VEC + q % VEC;
                  top.offer_many(hits && at < n * VEC ? score_key(to_f32(se[at]), x0 + at) : 0ull, k, lane);
                  hits &= hits - 1;
                }
                return;
              }
              // later mostly one lane with one entry: the 16 entries of two lanes a
              // round (4096 bf16 rows of 32000: 193 -> 187 us; alone it took rows of
              // 1000 from 76 to 95 us)
              const int q = lane % NE, mine = (warp * NV + q / VEC) * 32;
#pragma unroll 1
              while (reach) {
                const int l0 = __ffs(reach) - 1;
                reach &= reach - 1;
                const int l = lane < NE ? l0 : __ffs(reach) - 1;
                reach &= reach - 1;
                const int at = (mine + l) * VEC + q % VEC;
                unsigned long long key = 0ull;
                if (l >= 0 && at < n * VEC) {
                  const float v = to_f32(se[at]);
                  if (!(v < top.bar)) key = score_key(v, x0 + at);
                }
                top.offer_many(key, k, lane);
              }
            });
        }
        __syncwarp();
        if (lane == 0) tc5::mbar_arrive(&empty[sg]);
      }
      // head and tail: at most 2 (VEC - 1) < 32 entries, warp 0 of the first CTA
      if (part == 0 && warp == 0 && (head > 0 || tail0 < a.V)) {
        const int at = lane < 16 ? lane : tail0 + lane - 16;
        const bool ok = lane < 16 ? lane < head : at < a.V;
        float x[1] = {ok ? to_f32(src[at]) : -INFINITY};
        sums(x, x[0]);
        count(x, [&](int) { return at; }, [&](int) { return ok; });
        if (k > 0)
          pick(x[0], [&](unsigned) { top.offer_many(ok ? score_key(x[0], at) : 0ull, k, lane); });
      }

      // ---- warp, CTA and cluster merges
      st.reduce<32>(c);
      before = warp_sum_i(before);
      if (lane == 0) {
        wst[warp] = st;
        wbef[warp] = before;
      }
      consumers_sync();
      if (k > 0) {
        const float bar = cta_bar();
        if (top.list != 0ull && !(key_score(top.list) < bar)) s_keys[atomicAdd(&s_n, 1)] = top.list;
        consumers_sync();
      }
      if (warp == 0) {
        if (k > 0) {  // in any order: the keys are distinct
          top = WarpTop();
          const int n = *(volatile int*)&s_n;
#pragma unroll 1
          for (int i = 0; i < n; i += 32) top.offer_many(i + lane < n ? s_keys[i + lane] : 0ull, k, lane);
        }
        st = wst[lane & (kLpWarps - 1)];
        st.reduce<kLpWarps>(c);
        for (int w = 1; w < kLpWarps; ++w) before += wbef[w];
        if (C > 1) {
          *cluster.map_shared_rank(&cres[part][lane], 0) = top.list;
          if (lane == 0) {
            *cluster.map_shared_rank(&cst[part], 0) = st;
            *cluster.map_shared_rank(&cbef[part], 0) = before;
          }
        }
      }
      if (C > 1) cluster.sync();  // the partials have landed
      if (part == 0 && warp == 0 && !none && !bad) {
        for (int r = 1; r < C; ++r) {
          if (k > 0) top.merge(cres[r][lane], k, lane);
          st.merge(cst[r], c);
          before += cbef[r];
        }
        // a row without a finite maximum (every entry -inf) has no distribution
        const float ls = st.s > 0.0f ? logf(st.s) : NAN;
        if (lane == 0) {
          a.logprob[entry] = token >= 0 ? (xt - st.r) * tau - ls : NAN;
          if (a.entropy) a.entropy[entry] = ls - tau * st.w / st.s;
          if (a.rank) a.rank[entry] = token >= 0 ? before : -1;
        }
        if (lane < k) {
          const int id = (int)(~(uint32_t)(top.list & 0xffffffffull));
          if (a.top_tokens) a.top_tokens[entry * k + lane] = id;
          // after a timeout the list may be short
          if (a.top_logprobs)
            a.top_logprobs[entry * k + lane] = (unsigned)id < (unsigned)a.V ? (to_f32(src[id]) - st.r) * tau - ls : NAN;
        }
      }
    }
    if (part == 0 && warp == 0 && (none || bad)) {
      write_none(a, entry, lane);
      if (lane == 0 && bad) atomicOr(&a.status[b], bad);
    }
    chunks += n_chunks;
    if (item + step < entries) {  // the lists and partials are read before the next item writes its own
      if (C > 1) cluster.sync();
      else consumers_sync();
    }
  }
  __syncthreads();
  if (abort_flag && threadIdx.x == 0) {
    // a wait ran out: the CTA's own copies land before it exits, and every
    // request of the call may be short of a row
    for (int st = 0; st < kLpStages; ++st)
      if (s_last[st] >= 0) tc5::mbar_drain(&full[st], (s_last[st] / kLpStages) & 1);
    for (int b = 0; b < a.B; ++b) atomicOr(&a.status[b], SPEC_DEV_TIMEOUT);
  }
}

static spec_status launch_logprobs(LpArgs a, spec_dtype dtype, long long entries, cudaStream_t stream) {
  int sms = 0, dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return SPEC_ERR_CUDA;
  // a path call knows its rows on the device alone: five accepted nodes a request
  // stand for them (64 requests, V 32000: 29 us with C = 1, 37 with 2, 52 with 4;
  // 8 requests, V 128256: 48 us with C = 1, 25 with 8)
  a.live = a.path != nullptr && a.B <= kLpMaxLive;
  const long long rows = a.live ? std::min(entries, 5LL * a.B) : entries;
  int C = 1;
  while (C < kLpMaxCluster && rows * C * 6 <= 8LL * sms && a.V / (2 * C) >= 2048) C *= 2;
  const long long clusters = std::min<long long>(entries, std::max(1, 3 * sms / C));  // what the GPU holds at once
  a.C = C;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(clusters * C), 1, 1);
  cfg.blockDim = dim3(kLpThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.dynamicSmemBytes = kLpDyn;
  auto kern = dtype == SPEC_F32 ? logprobs_kernel<float> : logprobs_kernel<__nv_bfloat16>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kLpDyn);
  if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, kern, a, entries);
  if (e != cudaSuccess || cudaGetLastError() != cudaSuccess) return SPEC_ERR_CUDA;
  return SPEC_OK;
}

// Scalar checks of both calls (before any pointer is looked at).
static spec_status logprobs_check(int B, int T, int V, int k, spec_dtype dtype) {
  if (B < 0 || T < 0 || V <= 0 || k < 0) return SPEC_ERR_INVALID_ARG;
  if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_INVALID_ARG;
  if (k > V) return SPEC_ERR_INVALID_ARG;
  if (k > 32 || V > SPEC_MAX_VOCAB) return SPEC_ERR_UNSUPPORTED;
  return SPEC_OK;
}

}  // namespace spectree

using namespace spectree;

extern "C" {

spec_status spec_token_logprobs(const void* logits, spec_dtype dtype, const int32_t* tokens, const int32_t* seq_off,
                                const float* inv_temperature, int B, int T, int V, int k, float* logprob,
                                float* entropy, int32_t* rank, int32_t* top_tokens, float* top_logprobs,
                                int32_t* status, void* stream) {
  SPEC_NVTX_RANGE("spec_token_logprobs");
  const spec_status sc = logprobs_check(B, T, V, k, dtype);
  if (sc != SPEC_OK) return sc;
  if (B == 0 || T == 0) return SPEC_OK;
  if (!logits || !tokens || !seq_off || !logprob || !status) return SPEC_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(logits) & (dtype == SPEC_F32 ? 3 : 1)) != 0) return SPEC_ERR_INVALID_ARG;
  LpArgs a = {};
  a.logits = logits;
  a.tokens = tokens;
  a.off = seq_off;
  a.inv_temp = inv_temperature;
  a.logprob = logprob;
  a.entropy = entropy;
  a.rank = rank;
  a.top_tokens = top_tokens;
  a.top_logprobs = top_logprobs;
  a.status = status;
  a.B = B;
  a.T = T;
  a.V = V;
  a.k = top_tokens || top_logprobs ? k : 0;
  return launch_logprobs(a, dtype, T, (cudaStream_t)stream);
}

spec_status spec_path_logprobs(const void* p_logits, spec_dtype dtype, const int32_t* tree_off, const int32_t* path,
                               const int32_t* accept_len, const int32_t* emitted, const float* inv_temperature, int B,
                               int T, int n_max, int V, int k, float* logprob, float* entropy, int32_t* rank,
                               int32_t* top_tokens, float* top_logprobs, int32_t* status, void* stream) {
  SPEC_NVTX_RANGE("spec_path_logprobs");
  const spec_status sc = logprobs_check(B, T, V, k, dtype);
  if (sc != SPEC_OK) return sc;
  if (n_max < 0) return SPEC_ERR_INVALID_ARG;
  if (n_max > SPEC_MAX_NODES) return SPEC_ERR_UNSUPPORTED;
  if (B == 0 || n_max == 0) return SPEC_OK;
  if (!p_logits || !tree_off || !path || !accept_len || !emitted || !logprob || !status) return SPEC_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(p_logits) & (dtype == SPEC_F32 ? 3 : 1)) != 0) return SPEC_ERR_INVALID_ARG;
  LpArgs a = {};
  a.logits = p_logits;
  a.tokens = emitted;
  a.off = tree_off;
  a.path = path;
  a.accept_len = accept_len;
  a.inv_temp = inv_temperature;
  a.logprob = logprob;
  a.entropy = entropy;
  a.rank = rank;
  a.top_tokens = top_tokens;
  a.top_logprobs = top_logprobs;
  a.status = status;
  a.B = B;
  a.T = T;
  a.n_max = n_max;
  a.V = V;
  a.k = top_tokens || top_logprobs ? k : 0;
  return launch_logprobs(a, dtype, (long long)B * n_max, (cudaStream_t)stream);
}

}  // extern "C"
