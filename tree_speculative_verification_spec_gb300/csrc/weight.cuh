// Internal interface between the attention-weight host dispatch and its kernels.
#pragma once

#include "common.cuh"

namespace spectree {

// Rows are (counted token, query head of the group) pairs of one kv-head: row r
// of request b is counted token r / g, head kvh * g + r % g.  The counted tokens
// are the last `cnt` of the request's m (all, or the window); token i (from 0 in
// the request) sees slots 0 .. P + i and its queries are row off + i of q, or off
// + path[i] for an accepted path.
struct WeightArgs {
  const void* q;
  const void* k_cache;
  const int32_t* block_table;
  const int32_t* prefix_len;
  const int32_t* seq_off;
  const int32_t* path;        // NULL: packed rows
  const int32_t* accept_len;
  const float* before;        // NULL: zeros
  float* weight;
  int32_t* status;
  float2* ws_ml;              // [splits][Hkv][T * g][parts] partial (reference, sum) in the log2 domain, at (off + i) g + head of token i
  float* ws_part;             // [parts][B][Hkv][max_prefix + n_max] sums over a part of the rows (tensor cores, parts > 1)
  int parts;                  // of a request's rows, for the sums over many of them
  float* ws_lse;              // [Hkv][T * g] minus log2 of the whole sum (tensor cores)
  long long stride;           // floats of one (request, kv-head) of before and weight
  int path_stride, window;
  int max_blocks, block_size, num_blocks;
  int B, T, n_max, max_prefix, Hq, Hkv, D, g;
  int splits, chunk;          // split s of the statistics takes keys [s * chunk, (s + 1) * chunk)
  int per_req;                // row tiles per request (0: numbered along the packing, as in prompt.cuh)
  float scale_log2, decay;
};

// One request's share of a call; ok is false when it is left as it was.
struct WeightRequest {
  int b, off, n, m, cnt, P;
  bool ok;
};

// The SPEC_DEV_* bits of request b's own arguments, its path's entries left out.
__device__ __forceinline__ int weight_check(const WeightArgs& a, int b, WeightRequest& r) {
  r.b = b;
  r.off = a.seq_off[b];
  r.n = a.seq_off[b + 1] - r.off;
  r.P = a.prefix_len[b];
  r.m = a.path ? a.accept_len[b] : r.n;
  r.cnt = a.window > 0 ? min(r.m, a.window) : r.m;
  if (r.off < 0 || r.n < 0 || r.n > a.n_max || r.n > a.T - r.off) return SPEC_DEV_BAD_TREE;
  if (r.m < 0 || r.m > r.n || (a.path && r.m > a.path_stride)) return SPEC_DEV_BAD_PATH;
  const long long end = (long long)r.P + r.m;
  if (r.P < 0 || r.P > a.max_prefix || end > (long long)a.max_blocks * a.block_size || end > a.stride) return SPEC_DEV_CAPACITY;
  return 0;
}

// Whether entry i of the path (counted tokens only) names a row of the request.
__device__ __forceinline__ bool weight_path_bad(const WeightArgs& a, const WeightRequest& r, int i) {
  const int p = a.path[(size_t)r.b * a.path_stride + i];
  return p < 0 || p >= r.n;
}

// Row of q of token i.
__device__ __forceinline__ int weight_q_row(const WeightArgs& a, const WeightRequest& r, int i) {
  return r.off + (a.path ? a.path[(size_t)r.b * a.path_stride + i] : i);
}

// First row tile number of request b, with M rows a tile.
__device__ __forceinline__ long long weight_first_tile(const WeightArgs& a, int b, int M) {
  return a.per_req > 0 ? (long long)b * a.per_req : (long long)a.seq_off[b] * a.g / M + b;
}

// The request of row tile `tile`: the last one whose first tile is not above it.
__device__ __forceinline__ int weight_find(const WeightArgs& a, long long tile, int M) {
  if (a.per_req > 0) return (int)(tile / a.per_req);
  int lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (weight_first_tile(a, mid, M) <= tile) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Where the partial sums of counted token 0's first head lie, less the split's part.
__device__ __forceinline__ size_t weight_ws_row(const WeightArgs& a, int kvh, int off, int first) {
  return (size_t)kvh * a.T * a.g + (size_t)(off + first) * a.g;
}

// Two partial sums, (reference, sum) each, as one.
__device__ __forceinline__ float2 weight_join(float2 x, float2 y) {
  if (!(x.y > 0.0f)) return y;
  if (!(y.y > 0.0f)) return x;
  const float top = fmaxf(x.x, y.x);
  return make_float2(top, x.y * exp2f(x.x - top) + y.y * exp2f(y.x - top));
}

struct WeightPlan {
  int splits, chunk;
  long long tiles;  // row tiles, before heads and splits
};

cudaError_t launch_weight_tc(const WeightArgs& a, cudaStream_t stream);
cudaError_t launch_weight_cc(const WeightArgs& a, const WeightPlan& p, cudaStream_t stream);

}  // namespace spectree
