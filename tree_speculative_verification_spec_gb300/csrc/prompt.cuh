// Internal interface between the prompt-attention host dispatch and its kernels.
#pragma once

#include "common.cuh"

namespace spectree {

// Rows are (token, query head of the group) pairs of one kv-head: row r of
// request b is token r / g, head kvh * g + r % g.  Request b's row tiles are
// numbered from floor(seq_off[b] * g / M) + b: with M rows a tile, the gap to
// the next request's first tile is at least ceil(n_b * g / M), so tiles need
// no prefix sum over the batch and floor(T * g / M) + B of them cover every
// batch of T tokens.
struct PromptArgs {
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const int32_t* block_table;
  const int32_t* prefix_len;
  const int32_t* seq_off;
  void* out;
  int32_t* status;
  float* ws_o;   // [splits][T * Hq][D] partial outputs (unnormalised), fp32
  float* ws_ml;  // [splits][T * Hq][2] partial (reference, sum) in the log2 domain
  int max_blocks, block_size, num_blocks;
  int B, T, n_max, max_prefix, Hq, Hkv, D, g;
  int splits, chunk;  // split s takes keys [s * chunk, (s + 1) * chunk)
  float scale_log2;   // scale * log2(e)
};

// One request's share of a call; ok is false when it is not computed (its
// arguments are out of range, or it came in flagged).
struct PromptRequest {
  int b, off, n, P;
  bool ok;
};

// The SPEC_DEV_* bits of request b's own arguments.
__device__ __forceinline__ int prompt_check(const PromptArgs& a, int off, int n, int P) {
  if (off < 0 || n < 0 || n > a.n_max || n > a.T - off) return SPEC_DEV_BAD_TREE;
  if (P < 0 || P > a.max_prefix || (long long)P + n > (long long)a.max_blocks * a.block_size) return SPEC_DEV_CAPACITY;
  return 0;
}

__device__ __forceinline__ PromptRequest prompt_request(const PromptArgs& a, int b) {
  PromptRequest r;
  r.b = b;
  r.off = a.seq_off[b];
  r.n = a.seq_off[b + 1] - r.off;
  r.P = a.prefix_len[b];
  r.ok = prompt_check(a, r.off, r.n, r.P) == 0 && *(const volatile int32_t*)&a.status[b] == 0;
  return r;
}

// First tile number of request b.
__device__ __forceinline__ long long prompt_first_tile(const PromptArgs& a, int b, int M) {
  return (long long)a.seq_off[b] * a.g / M + b;
}

// The request of tile number `tile`: the last one whose first tile is not above it.
__device__ __forceinline__ int prompt_find(const PromptArgs& a, long long tile, int M) {
  int lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prompt_first_tile(a, mid, M) <= tile) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Flags every request whose own arguments are out of range: `count` threads of
// one CTA of a call do it; every CTA leaves such requests out.
__device__ __forceinline__ void prompt_flag_requests(const PromptArgs& a, int thread, int count) {
  for (int b = thread; b < a.B; b += count) {
    const int off = a.seq_off[b];
    const int bad = prompt_check(a, off, a.seq_off[b + 1] - off, a.prefix_len[b]);
    if (bad) atomicOr(&a.status[b], bad);
  }
}

constexpr int kPromptCcRows = 64;   // rows per CTA of the CUDA-core kernel
constexpr int kPromptTcRows = 256;  // rows per work item of the tensor-core kernel

struct PromptPlan {
  int splits, chunk;
  long long tiles;  // row tiles, before heads and splits
};

cudaError_t launch_prompt_cc(const PromptArgs& a, const PromptPlan& p, cudaStream_t stream);
cudaError_t launch_prompt_tc(const PromptArgs& a, const PromptPlan& p, cudaStream_t stream);

}  // namespace spectree
