// Prompt attention over the paged cache: fp32 kernel, split-key combine, and
// the host entry point.
//
// Row i of request b (packed at seq_off[b] + i) is the token at slot
// s = prefix_len[b] + i and sees slots 0 .. s:
//   out = sum_{k <= s} e^(scale q.K_k - m) V_k / sum_{k <= s} e^(scale q.K_k - m)
// for any reference m.  Keys are walked once with the running maximum as
// reference (online softmax in the log2 domain).
#include <algorithm>
#include <climits>
#include <cmath>

#include "prompt.cuh"

namespace spectree {

__device__ __forceinline__ float pr_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// CUDA-core kernel: a CTA takes 64 rows of one kv-head group and one key
// range, 64 keys at a time; 256 threads as 16 x 16, each 4 rows x 4 keys of
// the scores and 4 rows x D / 16 columns of the output.  Per 4 columns of q
// and K a thread reads 8 float4 for 64 multiply-adds, two to an instruction (the
// tensor cores have no fp32 product).  Shared memory is as busy as the FMA pipe:
// 4 x 700 tokens after 2000 (32/8 heads, D 128): 865 us, 31 TFLOP/s; one
// multiply-add an instruction 942 us.
constexpr int kPrThreads = 256;
constexpr int kPrRows = kPromptCcRows;
constexpr int kPrKeys = 64;

template <int D> struct PromptCcSmem {
  static constexpr int kStride = D + 4;  // 16-byte rows that start in other banks
  static constexpr int kPStride = kPrKeys + 4;
  float q[kPrRows * kStride];
  float k[kPrKeys * kStride];  // the probabilities [row][kPStride] after the scores
  float v[kPrKeys * D];
};

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }

template <int D>
__global__ void __launch_bounds__(kPrThreads, 2) prompt_cc_kernel(const PromptArgs a) {
  using S = PromptCcSmem<D>;
  extern __shared__ __align__(16) float dyn[];
  S& sm = *reinterpret_cast<S*>(dyn);
  __shared__ int s_badblk;
  const int kvh = blockIdx.z, split = blockIdx.y;
  if (blockIdx.x == 0 && split == 0 && kvh == 0) prompt_flag_requests(a, threadIdx.x, kPrThreads);
  // the last tiles of a request see the most keys: they start first
  const long long tile = (long long)gridDim.x - 1 - blockIdx.x;
  const int g = a.g;
  // one thread reads: the status word may change meanwhile, and every thread
  // of the CTA must take the same branch
  __shared__ PromptRequest s_rq;
  if (threadIdx.x == 0) s_rq = prompt_request(a, prompt_find(a, tile, kPrRows));
  __syncthreads();
  const PromptRequest rq = s_rq;
  if (!rq.ok) return;
  const long long mt = tile - prompt_first_tile(a, rq.b, kPrRows);
  const long long R = (long long)rq.n * g;
  if (mt < 0 || mt * kPrRows >= R) return;
  const int r0 = (int)(mt * kPrRows), rows = (int)min((long long)kPrRows, R - r0);
  const int k_begin = split * a.chunk;
  const int k_end = min(rq.P + (r0 + rows - 1) / g + 1, k_begin + a.chunk);
  if (k_begin >= k_end) return;

  const float* __restrict__ q = static_cast<const float*>(a.q);
  const float* __restrict__ kc = static_cast<const float*>(a.k_cache);
  const float* __restrict__ vc = static_cast<const float*>(a.v_cache);
  const int32_t* bt = a.block_table + (size_t)rq.b * a.max_blocks;
  const int bs = a.block_size;
  if (threadIdx.x == 0) s_badblk = 0;
  for (int i = threadIdx.x; i < kPrRows * (D / 4); i += kPrThreads) {
    const int r = i / (D / 4), c = (i % (D / 4)) * 4;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (r < rows) {
      const int t = rq.off + (r0 + r) / g, h = kvh * g + (r0 + r) % g;
      v = load4(q + ((size_t)t * a.Hq + h) * D + c);
    }
    *reinterpret_cast<float4*>(sm.q + r * S::kStride + c) = v;
  }

  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  constexpr int DJ = D / 64;  // float4 columns per thread: tx * 4 + 64 * jj
  float m[4], l[4];
  float2 o[4][DJ * 2];
  int last[4];  // the last key row i sees
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.0f;
    last[i] = rq.P + min(rq.n - 1, (r0 + ty * 4 + i) / g);
#pragma unroll
    for (int j = 0; j < DJ * 2; ++j) o[i][j] = make_float2(0.0f, 0.0f);
  }
  for (int k0 = k_begin; k0 < k_end; k0 += kPrKeys) {
    __syncthreads();
    for (int i = threadIdx.x; i < kPrKeys * (D / 4); i += kPrThreads) {
      const int kk = i / (D / 4), c = (i % (D / 4)) * 4, k = k0 + kk;
      float4 kv = make_float4(0.0f, 0.0f, 0.0f, 0.0f), vv = kv;
      if (k < k_end) {
        const int blk = bt[k / bs];
        if (blk < 0 || blk >= a.num_blocks) {
          s_badblk = 1;
        } else {
          const size_t base = (((size_t)blk * a.Hkv + kvh) * bs + k % bs) * D + c;
          kv = load4(kc + base);
          vv = load4(vc + base);
        }
      }
      *reinterpret_cast<float4*>(sm.k + kk * S::kStride + c) = kv;
      *reinterpret_cast<float4*>(sm.v + kk * D + c) = vv;
    }
    __syncthreads();
    float2 s2[4][4];  // even and odd pairs of columns
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s2[i][j] = make_float2(0.0f, 0.0f);
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
      float4 qa[4], kb[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) qa[i] = *reinterpret_cast<const float4*>(sm.q + (ty * 4 + i) * S::kStride + c);
#pragma unroll
      for (int j = 0; j < 4; ++j) kb[j] = *reinterpret_cast<const float4*>(sm.k + (tx + 16 * j) * S::kStride + c);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s2[i][j] = __ffma2_rn(make_float2(qa[i].x, qa[i].y), make_float2(kb[j].x, kb[j].y), s2[i][j]);
          s2[i][j] = __ffma2_rn(make_float2(qa[i].z, qa[i].w), make_float2(kb[j].z, kb[j].w), s2[i][j]);
        }
    }
    __syncthreads();  // the keys are read: their room takes the probabilities
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float mx = -INFINITY, s[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = k0 + tx + 16 * j;
        s[j] = k <= last[i] && k < k_end ? (s2[i][j].x + s2[i][j].y) * a.scale_log2 : -INFINITY;
        mx = fmaxf(mx, s[j]);
      }
#pragma unroll
      for (int w = 8; w; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
      const float mnew = fmaxf(m[i], mx);
      const float ref = mnew == -INFINITY ? 0.0f : mnew;  // nothing visible yet: every weight is 0
      const float alpha = pr_exp2(m[i] - ref);
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = pr_exp2(s[j] - ref);
        sum += p;
        sm.k[(ty * 4 + i) * S::kPStride + tx + 16 * j] = p;
      }
#pragma unroll
      for (int w = 8; w; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
      l[i] = l[i] * alpha + sum;
      m[i] = mnew;
#pragma unroll
      for (int j = 0; j < DJ * 2; ++j) o[i][j] = __fmul2_rn(o[i][j], make_float2(alpha, alpha));
    }
    __syncwarp();  // a warp's rows are its own: both halves of it wrote them
#pragma unroll 2
    for (int kk = 0; kk < kPrKeys; kk += 4) {
      float4 p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const float4*>(sm.k + (ty * 4 + i) * S::kPStride + kk);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float4 v[DJ];
#pragma unroll
        for (int jj = 0; jj < DJ; ++jj)
          v[jj] = *reinterpret_cast<const float4*>(sm.v + (kk + e) * D + tx * 4 + 64 * jj);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float w = e == 0 ? p[i].x : e == 1 ? p[i].y : e == 2 ? p[i].z : p[i].w;
#pragma unroll
          for (int jj = 0; jj < DJ; ++jj) {
            o[i][jj * 2] = __ffma2_rn(make_float2(w, w), make_float2(v[jj].x, v[jj].y), o[i][jj * 2]);
            o[i][jj * 2 + 1] = __ffma2_rn(make_float2(w, w), make_float2(v[jj].z, v[jj].w), o[i][jj * 2 + 1]);
          }
        }
      }
    }
  }
  __syncthreads();
  if (threadIdx.x == 0 && s_badblk) atomicOr(&a.status[rq.b], SPEC_DEV_BAD_BLOCK);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = ty * 4 + i;
    if (r >= rows) continue;
    const int t = rq.off + (r0 + r) / g, h = kvh * g + (r0 + r) % g;
    const size_t row = (size_t)t * a.Hq + h;
    if (a.splits == 1) {
      const float inv = 1.0f / l[i];
      float* out = static_cast<float*>(a.out) + row * D;
#pragma unroll
      for (int j = 0; j < DJ; ++j)
        *reinterpret_cast<float4*>(out + tx * 4 + 64 * j) =
            make_float4(o[i][j * 2].x * inv, o[i][j * 2].y * inv, o[i][j * 2 + 1].x * inv, o[i][j * 2 + 1].y * inv);
    } else {
      float* wo = a.ws_o + ((size_t)split * a.T * a.Hq + row) * D;
#pragma unroll
      for (int j = 0; j < DJ; ++j)
        *reinterpret_cast<float4*>(wo + tx * 4 + 64 * j) =
            make_float4(o[i][j * 2].x, o[i][j * 2].y, o[i][j * 2 + 1].x, o[i][j * 2 + 1].y);
      if (tx == 0) *reinterpret_cast<float2*>(a.ws_ml + ((size_t)split * a.T * a.Hq + row) * 2) = make_float2(m[i], l[i]);
    }
  }
}

// Split-key combine: out = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s over
// the splits that begin at or before the row's last key.  One warp per row:
// lane s holds split s's weight (32 splits at a time), and four splits' rows are
// loaded before any is added, since one row's chain of loads is all there is to
// wait for.  A programmatic dependent of the attention kernel.
template <typename T, int D>
__global__ void __launch_bounds__(256) prompt_combine_kernel(const PromptArgs a) {
  const long long row = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const long long rows = (long long)a.T * a.Hq;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the partial rows and the status are the attention's
  if (row >= rows) return;
  const int t = (int)(row / a.Hq);
  int lo = 0, hi = a.B;  // the last request with seq_off[lo] <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.seq_off[mid] <= t) lo = mid;
    else hi = mid;
  }
  const PromptRequest rq = prompt_request(a, lo);
  const int i = t - rq.off;
  if (!__shfl_sync(0xffffffffu, (int)rq.ok, 0) || i < 0 || i >= rq.n) return;  // one lane's word for the warp
  const int ns = min(a.splits, (rq.P + i) / a.chunk + 1);
  const float2* ml = reinterpret_cast<const float2*>(a.ws_ml) + row;
  float M = -INFINITY;
  for (int s = lane; s < ns; s += 32) M = fmaxf(M, ml[s * rows].x);
  M = warp_max_f(M);
  const float* os = a.ws_o + row * D + lane;
  float sum = 0.0f, acc[D / 32];
#pragma unroll
  for (int j = 0; j < D / 32; ++j) acc[j] = 0.0f;
  for (int s0 = 0; s0 < ns; s0 += 32) {
    const float2 x = s0 + lane < ns ? ml[(s0 + lane) * rows] : make_float2(-INFINITY, 0.0f);
    const float wl = x.x == -INFINITY ? 0.0f : pr_exp2(x.x - M);  // no visible key in the split
    sum = fmaf(wl, x.y, sum);
    const int n = min(32, ns - s0);
    for (int s = 0; s < n; s += 4) {
      float o[4][D / 32];
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int j = 0; j < D / 32; ++j) o[q][j] = s + q < n ? os[(s0 + s + q) * rows * D + 32 * j] : 0.0f;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float w = __shfl_sync(0xffffffffu, wl, (s + q) & 31);
#pragma unroll
        for (int j = 0; j < D / 32; ++j) acc[j] = s + q < n ? fmaf(w, o[q][j], acc[j]) : acc[j];
      }
    }
  }
  const float inv = 1.0f / warp_sum_f(sum);
  T* out = static_cast<T*>(a.out) + row * D;
#pragma unroll
  for (int j = 0; j < D / 32; ++j) out[lane + 32 * j] = from_f32<T>(acc[j] * inv);
}

template <int D>
static cudaError_t launch_cc(const PromptArgs& a, const PromptPlan& p, cudaStream_t stream) {
  const int dyn = (int)sizeof(PromptCcSmem<D>);
  const cudaError_t e = cudaFuncSetAttribute(prompt_cc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, dyn);
  if (e != cudaSuccess) return e;
  prompt_cc_kernel<D><<<dim3((unsigned)p.tiles, p.splits, a.Hkv), kPrThreads, dyn, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_prompt_cc(const PromptArgs& a, const PromptPlan& p, cudaStream_t stream) {
  return a.D == 64 ? launch_cc<64>(a, p, stream) : launch_cc<128>(a, p, stream);
}

static cudaError_t launch_prompt_combine(const PromptArgs& a, spec_dtype dt, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(((long long)a.T * a.Hq + 7) / 8), 1, 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void (*kern)(const PromptArgs) = dt == SPEC_F32 ? (a.D == 64 ? prompt_combine_kernel<float, 64> : prompt_combine_kernel<float, 128>)
                                                  : (a.D == 64 ? prompt_combine_kernel<__nv_bfloat16, 64>
                                                               : prompt_combine_kernel<__nv_bfloat16, 128>);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// Row tiles and key splits of a call.  Keys are split only when the row tiles
// alone leave SMs idle.
// CUDA cores: a 64-key step of one CTA takes 4 us and more of the FMA pipe, so
// splits go down to one step, as far as about two CTAs an SM (one token over 600
// keys: 78 us whole, 33 us by 128 keys, 25 us by 64; 2 x 500 tokens after 500:
// 119, 72, 74).
// Tensor cores (one CTA an SM): the split count of least waves x (4 us of
// set-up and output + 1.3 us per 128-key step) + 5 us for the combine (512
// tokens: 21 us whole, 29 us in two; one token over 16384: 33 us in 19).
// max_splits: what the caller's workspace holds.
constexpr long long kPlanSms = 152;  // a GB300's; the size query is a host call that needs no device
static PromptPlan prompt_plan(int B, int T, int n_max, int max_prefix, int Hq, int Hkv, bool bf16, long long max_splits) {
  PromptPlan p;
  const int g = Hq / Hkv;
  p.tiles = (long long)T * g / (bf16 ? kPromptTcRows : kPromptCcRows) + B;
  const long long units = p.tiles * Hkv, keys = (long long)max_prefix + n_max;
  long long splits = 1;
  if (units < kPlanSms && !bf16)
    splits = std::max(1LL, std::min({max_splits, (2 * kPlanSms + units - 1) / units, keys / kPrKeys}));
  if (units < kPlanSms && bf16) {
    double best = 1e300;
    const long long most = std::max(1LL, std::min({max_splits, 64LL, (keys + 127) / 128}));
    for (long long s = 1; s <= most; ++s) {
      const long long steps = ((keys + s - 1) / s + 127) / 128;
      const double cost = (double)((units * s + kPlanSms - 1) / kPlanSms) * (4.0 + 1.3 * (double)steps) + (s > 1 ? 5.0 : 0.0);
      if (cost < best * 0.97) {  // fewer splits on near-ties: less partial traffic
        best = cost;
        splits = s;
      }
    }
  }
  const long long tile = bf16 ? 128 : kPrKeys;
  const long long chunk = std::max(tile, ((keys + splits - 1) / splits + tile - 1) / tile * tile);
  p.chunk = (int)std::min<long long>(chunk, 1LL << 30);
  p.splits = (int)std::max(1LL, (keys + chunk - 1) / chunk);
  return p;
}

constexpr size_t kPromptWsMin = 256;

static size_t prompt_ws_bytes(const PromptPlan& p, int T, int Hq, int D) {
  if (p.splits <= 1) return 0;
  const size_t o = (size_t)p.splits * T * Hq * D * sizeof(float);
  return ((o + 255) & ~(size_t)255) + (size_t)p.splits * T * Hq * 2 * sizeof(float);
}
// The most splits whose partial rows fit into `bytes` (0 and 1: none do).
static long long prompt_ws_splits(size_t bytes, int T, int Hq, int D) {
  return bytes < 256 ? 0 : (long long)((bytes - 255) / ((size_t)T * Hq * (D + 2) * sizeof(float)));
}

static spec_status prompt_shape_check(int B, int T, int n_max, int max_prefix, int Hq, int Hkv, int D,
                                      int block_size) {
  if (B < 0 || T < 0 || n_max < 0 || max_prefix < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0) return SPEC_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return SPEC_ERR_UNSUPPORTED;
  if (block_size < 8 || block_size > 65536 || (block_size & (block_size - 1))) return SPEC_ERR_UNSUPPORTED;
  if (B > 65535 || Hkv > 65535 || (long long)n_max * (Hq / Hkv) >= (1LL << 30) || (long long)max_prefix + n_max >= (1LL << 30))
    return SPEC_ERR_UNSUPPORTED;
  if ((long long)T * (Hq / Hkv) / kPrRows + B >= (1LL << 24) || (long long)T * Hq >= (1LL << 31))
    return SPEC_ERR_UNSUPPORTED;
  return SPEC_OK;
}

}  // namespace spectree

using namespace spectree;

extern "C" {

size_t spec_prompt_workspace_size(int B, int T, int n_max, int max_prefix, int Hq, int Hkv, int D) {
  if (B <= 0 || T <= 0 || n_max <= 0 || prompt_shape_check(B, T, n_max, max_prefix, Hq, Hkv, D, 16) != SPEC_OK)
    return kPromptWsMin;
  size_t best = kPromptWsMin;
  for (bool bf16 : {false, true})
    best = std::max(best, prompt_ws_bytes(prompt_plan(B, T, n_max, max_prefix, Hq, Hkv, bf16, INT_MAX), T, Hq, D));
  return best;
}

spec_status spec_prompt_attention(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                                  int max_blocks, int block_size, int num_blocks, const int32_t* prefix_len,
                                  const int32_t* seq_off, int B, int T, int n_max, int max_prefix, int Hq, int Hkv,
                                  int D, spec_dtype dtype, float scale, void* out, void* workspace,
                                  size_t workspace_bytes, int32_t* status, void* stream) {
  SPEC_NVTX_RANGE("spec_prompt_attention");
  if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_INVALID_ARG;
  if (!(scale >= 0.0f && scale < INFINITY)) return SPEC_ERR_INVALID_ARG;  // the largest score is the largest product
  const spec_status sc = prompt_shape_check(B, T, n_max, max_prefix, Hq, Hkv, D, block_size);
  if (sc != SPEC_OK) return sc;
  if (B == 0 || T == 0 || n_max == 0) return SPEC_OK;
  if (!q || !k_cache || !v_cache || !block_table || !prefix_len || !seq_off || !out || !status || max_blocks <= 0 ||
      num_blocks <= 0)
    return SPEC_ERR_INVALID_ARG;
  if (((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k_cache) | reinterpret_cast<uintptr_t>(v_cache) |
        reinterpret_cast<uintptr_t>(out)) & 15) != 0)
    return SPEC_ERR_INVALID_ARG;
  // the tensor-core path names cache rows by 32-bit coordinates, and items by a grid index
  if (dtype == SPEC_BF16 && (long long)num_blocks * Hkv * block_size >= (long long)INT32_MAX) return SPEC_ERR_UNSUPPORTED;
  PromptPlan plan = prompt_plan(B, T, n_max, max_prefix, Hq, Hkv, dtype == SPEC_BF16, INT_MAX);
  if (plan.tiles * Hkv * plan.splits > (long long)INT32_MAX) return SPEC_ERR_UNSUPPORTED;
  size_t need = prompt_ws_bytes(plan, T, Hq, D);
  if (need > 0 && (!workspace || workspace_bytes < kPromptWsMin || (reinterpret_cast<uintptr_t>(workspace) & 15)))
    return SPEC_ERR_WORKSPACE;
  if (workspace_bytes < need) {
    // a buffer that was sized for another batch: the best plan that fits it (with
    // whole keys in the end, which needs none)
    plan = prompt_plan(B, T, n_max, max_prefix, Hq, Hkv, dtype == SPEC_BF16, prompt_ws_splits(workspace_bytes, T, Hq, D));
    need = prompt_ws_bytes(plan, T, Hq, D);
  }
  PromptArgs a = {};
  a.q = q;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.block_table = block_table;
  a.prefix_len = prefix_len;
  a.seq_off = seq_off;
  a.out = out;
  a.status = status;
  if (need > 0) {
    const size_t o = (size_t)plan.splits * T * Hq * D * sizeof(float);
    a.ws_o = static_cast<float*>(workspace);
    a.ws_ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + ((o + 255) & ~(size_t)255));
  }
  a.max_blocks = max_blocks;
  a.block_size = block_size;
  a.num_blocks = num_blocks;
  a.B = B;
  a.T = T;
  a.n_max = n_max;
  a.max_prefix = max_prefix;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.D = D;
  a.g = Hq / Hkv;
  a.splits = plan.splits;
  a.chunk = plan.chunk;
  // The tensor-core kernel hides a key by -inf before the scaling, and -inf * 0 is
  // NaN: the smallest float stands for a scale of 0 (the largest finite score
  // times it is 2^-21, a weight of 1 + 3e-7).
  a.scale_log2 = std::max(scale * 1.4426950408889634f, 0x1p-149f);
  cudaStream_t st = (cudaStream_t)stream;
  if (need > 0) spec_workspace_canary(workspace, need, st);
  const cudaError_t e = dtype == SPEC_BF16 ? launch_prompt_tc(a, plan, st) : launch_prompt_cc(a, plan, st);
  if (e != cudaSuccess) return SPEC_ERR_CUDA;
  if (plan.splits > 1 && launch_prompt_combine(a, dtype, st) != cudaSuccess) return SPEC_ERR_CUDA;
  return SPEC_OK;
}

}  // extern "C"
