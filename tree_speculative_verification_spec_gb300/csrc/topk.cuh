// Ranking of scores and a warp's running top-k, shared by the tree builder's
// expansion level and the log-probability kernels: larger score first, equal
// scores by lower token id, NaN after every number, -0 equal to +0.
#pragma once

#include "common.cuh"

namespace spectree {

// Rank key of a draft score: larger is better.  High word: the float made
// orderable as an unsigned integer (-0 counted as +0, NaN below -inf); low
// word: the complement of the token id, so that equal scores rank the lower
// id first.  Keys of distinct tokens are distinct and all above 0.
__device__ __forceinline__ unsigned long long score_key(float v, int id) {
  uint32_t u = __float_as_uint(v);
  uint32_t k;
  if (v != v) {
    k = 0u;
  } else {
    if (u == 0x80000000u) u = 0u;
    k = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  }
  return ((unsigned long long)k << 32) | (unsigned long long)(~(uint32_t)id);
}

// The score of a key's high word: the bar below which no entry can enter a
// full list (-inf while the list has room or holds a NaN entry).
__device__ __forceinline__ float key_score(unsigned long long key) {
  const uint32_t k = (uint32_t)(key >> 32);
  if (k == 0u) return -INFINITY;
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// A warp's running top-k (k <= 32): lane r < k holds the r-th best key
// (descending), lanes >= k hold 0.  thr = the k-th best key (0 while there is
// room), bar = its score.
struct WarpTop {
  unsigned long long list = 0ull, thr = 0ull;
  float bar = -INFINITY;
  float floor = -INFINITY;  // a lower bound of the k-th best score, from a first sample

  // The (n + 1)-th largest of one value per lane (NaN counted as -inf), by a
  // bitonic sort across the warp.
  static __device__ __forceinline__ float nth_largest(float v, int n, int lane) {
    if (v != v) v = -INFINITY;
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1) {
#pragma unroll
      for (int stride = size >> 1; stride > 0; stride >>= 1) {
        const float o = __shfl_xor_sync(0xffffffffu, v, stride);
        const bool desc = ((lane & size) == 0) == ((lane & stride) == 0);  // keep the larger in the lower lane
        v = desc ? fmaxf(v, o) : fminf(v, o);
      }
    }
    return __shfl_sync(0xffffffffu, v, n);
  }

  // Lower bound for the bar from one sample per lane (its best score of a
  // first batch): the k-th largest of these 32 distinct entries.  No entry
  // scored below it can be among the k best.
  __device__ __forceinline__ void seed(float lane_best, int k, int lane) {
    floor = nth_largest(lane_best, k - 1, lane);
    bar = fmaxf(bar, floor);
  }

  // Inserts `key` (the same value in every lane) if it beats the k-th best.
  __device__ __forceinline__ void insert(unsigned long long key, int k, int lane) {
    if (key <= thr) return;  // warp-uniform
    const int pos = __popc(__ballot_sync(0xffffffffu, list > key));  // the greater keys are lanes 0 .. pos-1
    const unsigned long long up = __shfl_up_sync(0xffffffffu, list, 1);
    if (lane > pos) list = up;
    else if (lane == pos) list = key;
    if (lane >= k) list = 0ull;
    thr = __shfl_sync(0xffffffffu, list, k - 1);
    bar = fmaxf(key_score(thr), floor);
  }

  // Every lane offers one score (valid lanes only); called by the whole warp.
  __device__ __forceinline__ void offer(float v, int x, bool valid, int k, int lane) {
    unsigned m = __ballot_sync(0xffffffffu, valid && !(v < bar));
    while (m) {
      const int l = __ffs(m) - 1;
      m &= m - 1;
      insert(score_key(__shfl_sync(0xffffffffu, v, l), __shfl_sync(0xffffffffu, x, l)), k, lane);
    }
  }

  // Takes another list, sorted the same way (lane r the r-th best, 0 = nothing).
  // The larger of list[i] and other[31 - i] are the 32 best of both and rise
  // then fall, which five exchange steps sort: some 300 cycles, where an
  // insertion costs about 100 for each key.
  __device__ __forceinline__ void merge(unsigned long long other, int k, int lane) {
    const unsigned long long o = __shfl_sync(0xffffffffu, other, 31 - lane);
    list = list > o ? list : o;
#pragma unroll
    for (int stride = 16; stride > 0; stride >>= 1) {
      const unsigned long long y = __shfl_xor_sync(0xffffffffu, list, stride);
      list = ((lane & stride) == 0) == (y > list) ? y : list;
    }
    if (lane >= k) list = 0ull;
    thr = __shfl_sync(0xffffffffu, list, k - 1);
    bar = fmaxf(key_score(thr), floor);
  }

  // Every lane offers one key (0 = nothing); few are inserted, many are sorted
  // and merged.
  __device__ __forceinline__ void offer_many(unsigned long long key, int k, int lane) {
    unsigned m = __ballot_sync(0xffffffffu, key > thr);
    if (__popc(m) > 8) {
      unsigned long long v = key > thr ? key : 0ull;
#pragma unroll
      for (int size = 2; size <= 32; size <<= 1) {
#pragma unroll
        for (int stride = size >> 1; stride > 0; stride >>= 1) {
          const unsigned long long y = __shfl_xor_sync(0xffffffffu, v, stride);
          const bool desc = ((lane & size) == 0) == ((lane & stride) == 0);  // keep the larger in the lower lane
          v = desc == (y > v) ? y : v;
        }
      }
      merge(v, k, lane);
      return;
    }
    while (m) {
      const int l = __ffs(m) - 1;
      m &= m - 1;
      insert(__shfl_sync(0xffffffffu, key, l), k, lane);
    }
  }

  // Every lane offers one key (0 = nothing).
  __device__ __forceinline__ void offer_key(unsigned long long key, int k, int lane) {
    unsigned m = __ballot_sync(0xffffffffu, key > thr);
    while (m) {
      const int l = __ffs(m) - 1;
      m &= m - 1;
      insert(__shfl_sync(0xffffffffu, key, l), k, lane);
    }
  }
};

}  // namespace spectree
