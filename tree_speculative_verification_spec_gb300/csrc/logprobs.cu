// Log probabilities of given tokens, with the entropy of their distribution,
// the token's rank and the top alternatives.
//
// For one row of logits x, inverse temperature tau and given token t, with
// m = max x and d_i = x_i - m:
//   S = sum_i e^(tau d_i),  W = sum_i e^(tau d_i) d_i
//   log p(t) = tau d_t - log S
//   H = -sum_i p_i log p_i = log S - tau W / S
//   rank(t) = number of tokens ranked before t (larger logit, equal logits by
//             lower id, NaN last)
// Every value comes from one read of the row: each thread keeps (m, S, W)
// against its own running maximum, rescaled by 2^((m_old - m_new) tau log2 e)
// once per batch of loads that raises it, and the partials merge by the same
// rule across the warp, the CTA and the row's cluster.  The row is the only
// traffic that counts (V entries against a few words of results), so the
// kernel is bound by HBM for many rows and by launch and one row's latency
// for few.  One cluster of C CTAs per row: C = 1 when the rows alone fill the
// GPU, else enough CTAs to spread a row, with at least 2048 entries each.
#include <algorithm>

#include <cooperative_groups.h>

#include "topk.cuh"

namespace cg = cooperative_groups;

namespace spectree {

constexpr int kLpThreads = 256;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpMaxCluster = 8;
constexpr int kLpBatch = 4;  // 16-byte loads per thread issued before any is used

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

// Softmax statistics against a reference m: s = sum e^(tau (x - m)), w = sum
// e^(tau (x - m)) (x - m).  m = -inf: nothing (finite) seen yet.  A NaN stays
// NaN through every merge.
struct SoftStats {
  float m = -INFINITY, s = 0.0f, w = 0.0f;

  // the same sums against a larger reference (c = tau * log2 e)
  __device__ __forceinline__ void raise(float to, float c) {
    if (m == to) return;
    if (m == -INFINITY) {
      s = w = 0.0f;
    } else {
      const float delta = m - to;  // <= 0; -inf when `to` is +inf
      const float f = lp_exp2(delta * c);
      // e^(tau delta) vanishes faster than delta grows: the clamp keeps 0 * inf out
      w = f * fmaf(s, max_nan(delta, -1e30f), w);
      s *= f;
    }
    m = to;
  }
  __device__ __forceinline__ void merge(SoftStats o, float c) {
    const float to = max_nan(m, o.m);
    raise(to, c);
    o.raise(to, c);
    s += o.s;
    w += o.w;
  }
  __device__ __forceinline__ void add(float x, float c) {
    const float d = max_nan(x - m, -3e38f);  // -inf entries weigh nothing: e is 0, and 0 * d stays 0
    const float e = lp_exp2(d * c);
    s += e;
    w = fmaf(e, d, w);
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

__device__ __forceinline__ uint32_t rank_word(float v) { return (uint32_t)(score_key(v, 0) >> 32); }

template <typename T>
__global__ void __launch_bounds__(kLpThreads) logprobs_kernel(const LpArgs a) {
  constexpr int VEC = 16 / sizeof(T);
  __shared__ unsigned long long wres[kLpWarps][32];
  __shared__ unsigned long long cres[kLpMaxCluster][32];  // leader: the CTAs' lists
  __shared__ SoftStats wst[kLpWarps], cst[kLpMaxCluster];
  __shared__ int wbef[kLpWarps], cbef[kLpMaxCluster];
  cg::cluster_group cluster = cg::this_cluster();
  const int C = a.C, part = (int)cluster.block_rank();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long entry = blockIdx.x / C;  // the same for every CTA of the cluster
  const int k = a.k;

  // ---- the entry's row, request and token
  int b, token, bad = 0;
  long long row = 0;
  bool none = false;  // nothing to compute: the outputs say so
  if (a.path) {
    b = (int)(entry / a.n_max);
    const int i = (int)(entry % a.n_max);
    const int n_acc = a.accept_len[b];
    const int off = a.off[b], n = a.off[b + 1] - off;
    token = -1;
    none = i >= n_acc;
    if (n_acc > a.n_max) {
      none = true;
      bad = SPEC_DEV_BAD_PATH;
    }
    if (!none) {
      const int p = a.path[entry];
      token = a.tokens[entry];
      if (off < 0 || n < 0 || n > a.T - off || p < 0 || p >= n) bad |= SPEC_DEV_BAD_PATH;
      if (token < 0 || token >= a.V) bad |= SPEC_DEV_BAD_TOKEN;
      row = (long long)off + p;
    }
  } else {
    int lo = 0, hi = a.B;  // the last request with off[lo] <= entry
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.off[mid] <= entry) lo = mid;
      else hi = mid;
    }
    b = lo;
    row = entry;
    none = entry < a.off[b] || entry >= a.off[b + 1];  // a row no request owns
    token = none ? -1 : a.tokens[entry];
    if (token < -1 || token >= a.V) bad = SPEC_DEV_BAD_TOKEN;
  }
  float tau = 1.0f;
  if (!none && a.inv_temp) {
    tau = a.inv_temp[b];
    if (!(tau >= 1e-30f && tau < INFINITY)) bad |= SPEC_DEV_BAD_TEMP;
  }
  if (none || bad) {
    if (part == 0) {
      if (threadIdx.x == 0) {
        if (a.logprob) a.logprob[entry] = NAN;
        if (a.entropy) a.entropy[entry] = NAN;
        if (a.rank) a.rank[entry] = -1;
        if (bad && a.status) atomicOr(&a.status[b], bad);
      }
      if (threadIdx.x < k) {
        if (a.top_tokens) a.top_tokens[entry * k + threadIdx.x] = -1;
        if (a.top_logprobs) a.top_logprobs[entry * k + threadIdx.x] = NAN;
      }
    }
    return;  // the whole cluster leaves
  }

  const T* src = static_cast<const T*>(a.logits) + row * a.V;
  const float c = tau * 1.4426950408889634f;
  const float xt = token >= 0 ? to_f32(src[token]) : 0.0f;
  const uint32_t rt = rank_word(xt);

  // the row: a head up to the first 16-byte boundary, 16-byte vectors, a tail
  const int mis = (int)((reinterpret_cast<uintptr_t>(src) & 15) / sizeof(T));
  const int head = min(a.V, mis ? VEC - mis : 0);
  const int nvec = (a.V - head) / VEC;
  const int tail0 = head + nvec * VEC;
  const uint4* vec = reinterpret_cast<const uint4*>(src + head);
  const int per = (nvec + C - 1) / C;
  const int v0 = min(nvec, part * per), v1 = min(nvec, v0 + per);

  SoftStats st;
  WarpTop top;
  int before = 0;
  bool seeded = false;
  // one batch of N values per lane; value q of the lane has id `id(q)`, lanes beyond the
  // batch hold -inf at an id that `in(q)` tells apart
  auto consume = [&](auto& x, auto id, auto in) {
    constexpr int N = sizeof(x) / sizeof(float);
    float mx = -INFINITY;
#pragma unroll
    for (int q = 0; q < N; ++q) mx = max_nan(mx, x[q]);
    if (!(mx <= st.m)) st.raise(mx, c);
    if (st.m != -INFINITY) {
#pragma unroll
      for (int q = 0; q < N; ++q) st.add(x[q], c);
    }
    if (token >= 0) {
#pragma unroll
      for (int q = 0; q < N; ++q) {
        const uint32_t r = rank_word(x[q]);
        before += in(q) && (r > rt || (r == rt && id(q) < token));
      }
    }
    if (k > 0) {
      if (!seeded) {
        top.seed(mx, k, lane);
        seeded = true;
      }
      if (__any_sync(0xffffffffu, !(mx < top.bar))) {
#pragma unroll
        for (int q = 0; q < N; ++q) top.offer(x[q], id(q), in(q), k, lane);
      }
    }
  };
  for (int j0 = v0 + warp * kLpBatch * 32; j0 < v1; j0 += kLpWarps * kLpBatch * 32) {
    uint4 raw[kLpBatch];
#pragma unroll
    for (int q = 0; q < kLpBatch; ++q) {
      const int j = j0 + q * 32 + lane;
      if (j < v1) raw[q] = __ldcs(vec + j);
    }
    float x[kLpBatch * VEC];
#pragma unroll
    for (int q = 0; q < kLpBatch; ++q) {
      float y[VEC];
      lp_unpack<T>(raw[q], y);
      const bool ok = j0 + q * 32 + lane < v1;
#pragma unroll
      for (int e = 0; e < VEC; ++e) x[q * VEC + e] = ok ? y[e] : -INFINITY;
    }
    consume(
        x, [&](int q) { return head + (j0 + (q / VEC) * 32 + lane) * VEC + q % VEC; },
        [&](int q) { return j0 + (q / VEC) * 32 + lane < v1; });
  }
  // head and tail: at most 2 (VEC - 1) < 32 entries, warp 0 of the first CTA
  if (part == 0 && warp == 0 && (head > 0 || tail0 < a.V)) {
    const int at = lane < 16 ? lane : tail0 + lane - 16;
    const bool ok = lane < 16 ? lane < head : at < a.V;
    float x[1] = {ok ? to_f32(src[at]) : -INFINITY};
    consume(x, [&](int) { return at; }, [&](int) { return ok; });
  }

  // ---- warp, CTA and cluster merges
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    SoftStats y;
    y.m = __shfl_xor_sync(0xffffffffu, st.m, o);
    y.s = __shfl_xor_sync(0xffffffffu, st.s, o);
    y.w = __shfl_xor_sync(0xffffffffu, st.w, o);
    st.merge(y, c);
  }
  before = warp_sum_i(before);
  wres[warp][lane] = top.list;
  if (lane == 0) {
    wst[warp] = st;
    wbef[warp] = before;
  }
  __syncthreads();
  if (warp == 0) {
    for (int w = 1; w < kLpWarps; ++w) {
      if (k > 0) top.offer_key(wres[w][lane], k, lane);
      st.merge(wst[w], c);
      before += wbef[w];
    }
    if (C > 1) {
      *cluster.map_shared_rank(&cres[part][lane], 0) = top.list;
      if (lane == 0) {
        *cluster.map_shared_rank(&cst[part], 0) = st;
        *cluster.map_shared_rank(&cbef[part], 0) = before;
      }
    }
  }
  if (C > 1) cluster.sync();  // the partials have landed; no CTA touches another's memory after this
  if (part != 0 || warp != 0) return;
  for (int r = 1; r < C; ++r) {
    if (k > 0) top.offer_key(cres[r][lane], k, lane);
    st.merge(cst[r], c);
    before += cbef[r];
  }
  // a row without a finite maximum (every entry -inf) has no distribution
  const float ls = st.s > 0.0f ? logf(st.s) : NAN;
  if (lane == 0) {
    if (a.logprob) a.logprob[entry] = token >= 0 ? (xt - st.m) * tau - ls : NAN;
    if (a.entropy) a.entropy[entry] = ls - tau * st.w / st.s;
    if (a.rank) a.rank[entry] = token >= 0 ? before : -1;
  }
  if (lane < k) {
    const int id = (int)(~(uint32_t)(top.list & 0xffffffffull));
    if (a.top_tokens) a.top_tokens[entry * k + lane] = id;
    if (a.top_logprobs) a.top_logprobs[entry * k + lane] = (to_f32(src[id]) - st.m) * tau - ls;
  }
}

static spec_status launch_logprobs(LpArgs a, spec_dtype dtype, long long entries, cudaStream_t stream) {
  int sms = 0, dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return SPEC_ERR_CUDA;
  int C = 1;
  while (C < kLpMaxCluster && entries * C < 2LL * sms && a.V / (2 * C) >= 2048) C *= 2;
  if (entries * C >= (1LL << 31)) return SPEC_ERR_UNSUPPORTED;
  a.C = C;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(entries * C), 1, 1);
  cfg.blockDim = dim3(kLpThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = dtype == SPEC_F32 ? cudaLaunchKernelEx(&cfg, logprobs_kernel<float>, a)
                                          : cudaLaunchKernelEx(&cfg, logprobs_kernel<__nv_bfloat16>, a);
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
