// The attention weight that cached slots gather: host dispatch, and the
// CUDA-core kernels (fp32; the tensor cores take bf16 alone).
//
//   weight[b][h][s] = decay before[b][h][s] + sum over rows softmax(scale q K^T)[row][s]
//
// A column sum of a softmax needs every row's maximum and sum first, so there
// are two passes over the scores: statistics (row tiles against all keys, split
// over the keys when there are few rows) and sums (key tiles against the rows
// that see them).  Each slot's weight is one thread's sum in a fixed order: no
// atomics, the same bits every time.
#include <algorithm>
#include <climits>

#include "weight.cuh"

namespace spectree {

constexpr int kWtRows = 64, kWtFewRows = 16, kWtKeys = 64, kWtThreads = 256, kWtPad = 4;
// Rows per item of the tensor-core kernel: two tiles of the whole tokens of 128 rows.
static int weight_tc_rows(int g) { return g <= 128 ? 2 * (128 / g * g) : 256; }
constexpr int kWtParts = 2;     // partial sums it leaves of a row and split

// Loads a tile of N vectors transposed into shared memory as fp32, [D][64 + pad];
// `row(i)` gives the address of vector i, or NULL for zeros.  A warp takes 64 bytes
// of 8 vectors: whole sectors to read, two banks' conflict to write (a vector a
// warp wrote to two banks alone).
template <typename T, int D, int N, typename F>
__device__ __forceinline__ void load_tile(float* dst, F row) {
  constexpr int V = 16 / sizeof(T), C = D / V;
  const int lane = threadIdx.x & 31;
  for (int j = threadIdx.x / 32; j < N / 8 * (C / 4); j += kWtThreads / 32) {
    const int i = j % (N / 8) * 8 + (lane & 7), c = j / (N / 8) * 4 + (lane >> 3);
    const T* p = row(i);
    uint4 u = make_uint4(0, 0, 0, 0);
    if (p) u = *reinterpret_cast<const uint4*>(p + c * V);
    const T* x = reinterpret_cast<const T*>(&u);
#pragma unroll
    for (int e = 0; e < V; ++e) dst[(c * V + e) * (64 + kWtPad) + i] = to_f32(x[e]);
  }
}

// RT x 4 scores of this thread: rows RT ty .., keys 4 tx ..
template <int D, int RT>
__device__ __forceinline__ void scores(const float* q, const float* k, int ty, int tx, float (&s)[RT][4]) {
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[i][j] = 0.0f;
#pragma unroll 4
  for (int d = 0; d < D; ++d) {
    float xs[RT];
    if (RT == 4) *reinterpret_cast<float4*>(xs) = *reinterpret_cast<const float4*>(q + d * (64 + kWtPad) + 4 * ty);
    else xs[0] = q[d * (64 + kWtPad) + ty];
    const float4 y = *reinterpret_cast<const float4*>(k + d * (64 + kWtPad) + 4 * tx);
    const float ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = fmaf(xs[i], ys[j], s[i][j]);
  }
}

// Whether request b counts (the same answer in every thread of the CTA).
__device__ __forceinline__ bool weight_request_cta(const WeightArgs& a, int b, WeightRequest& r, bool flag) {
  __shared__ int s_status;
  const int bad = weight_check(a, b, r);
  if (threadIdx.x == 0) s_status = *(const volatile int32_t*)&a.status[b];
  __syncthreads();
  r.ok = bad == 0 && s_status == 0;
  int pb = 0;
  if (r.ok && a.path)
    for (int i = r.m - r.cnt + threadIdx.x; i < r.m; i += kWtThreads) pb |= weight_path_bad(a, r, i);
  pb = __syncthreads_or(pb);
  if (pb) r.ok = false;
  if (flag && threadIdx.x == 0 && (bad || pb)) atomicOr(&a.status[b], bad ? bad : SPEC_DEV_BAD_PATH);
  return r.ok;
}

template <typename T>
__device__ __forceinline__ const T* key_row(const WeightArgs& a, const int32_t* bt, int kvh, int s, int* bad) {
  const int blk = bt[s / a.block_size];
  if (blk < 0 || blk >= a.num_blocks) {
    *bad = 1;
    return nullptr;
  }
  return static_cast<const T*>(a.k_cache) + (((size_t)blk * a.Hkv + kvh) * a.block_size + s % a.block_size) * a.D;
}

// RT rows a thread: 64 rows a tile, or 16 where no request has more.
template <typename T, int D, int RT>
__global__ void __launch_bounds__(kWtThreads) weight_stats_cc_kernel(const WeightArgs a) {
  constexpr int ROWS = 16 * RT;
  extern __shared__ float sm[];
  float *sq = sm, *sk = sm + D * (64 + kWtPad);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int kvh = blockIdx.x % a.Hkv, split = blockIdx.x / a.Hkv % a.splits;
  const long long tile = blockIdx.x / a.Hkv / a.splits;
  const int b = weight_find(a, tile, ROWS);
  WeightRequest r;
  if (!weight_request_cta(a, b, r, false)) return;
  const long long at = tile - weight_first_tile(a, b, ROWS);
  const int R = r.cnt * a.g;
  if (at < 0 || at * ROWS >= R) return;
  const int r0 = (int)at * ROWS, first = r.m - r.cnt;
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  load_tile<T, D, ROWS>(sq, [&](int i) -> const T* {
    if (r0 + i >= R) return nullptr;
    return static_cast<const T*>(a.q) + ((size_t)weight_q_row(a, r, first + (r0 + i) / a.g) * a.Hq + kvh * a.g + (r0 + i) % a.g) * D;
  });
  const int last = first + (min(r0 + ROWS, R) - 1) / a.g;  // the tile's last token
  const int begin = split * a.chunk, end = min(begin + a.chunk, r.P + last + 1);
  const int32_t* bt = a.block_table + (size_t)b * a.max_blocks;
  float m[RT], l[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) m[i] = -INFINITY, l[i] = 0.0f;
  int bad = 0;
  for (int k0 = begin; k0 < end; k0 += kWtKeys) {
    __syncthreads();
    load_tile<T, D, kWtKeys>(sk, [&](int i) -> const T* { return k0 + i < end ? key_row<T>(a, bt, kvh, k0 + i, &bad) : nullptr; });
    __syncthreads();
    float s[RT][4];
    scores<D, RT>(sq, sk, ty, tx, s);
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int seen = r.P + first + (r0 + RT * ty + i) / a.g;  // the last slot this row sees
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = k0 + 4 * tx + j;
        s[i][j] = k < end && k <= seen ? s[i][j] * a.scale_log2 : -INFINITY;
        top = fmaxf(top, s[i][j]);
      }
#pragma unroll
      for (int o = 8; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      top = fmaxf(top, m[i]);
      if (top == -INFINITY) continue;  // the 16 lanes of a row agree
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) sum += exp2f(s[i][j] - top);
      l[i] = l[i] * exp2f(m[i] - top) + sum;
      m[i] = top;
    }
  }
#pragma unroll
  for (int i = 0; i < RT; ++i) {
#pragma unroll
    for (int o = 8; o; o >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
    const int row = r0 + RT * ty + i;
    if (tx == 0 && row < R)
      a.ws_ml[(size_t)split * a.T * a.Hq + weight_ws_row(a, kvh, r.off, first) + row] = make_float2(m[i], l[i]);
  }
  if (bad) atomicOr(&a.status[b], SPEC_DEV_BAD_BLOCK);
}

template <typename T, int D, int RT>
__global__ void __launch_bounds__(kWtThreads) weight_sums_cc_kernel(const WeightArgs a, int key_tiles) {
  constexpr int ROWS = 16 * RT;
  extern __shared__ float sm[];
  float *sq = sm, *sk = sm + D * (64 + kWtPad);
  __shared__ float s_lse[ROWS], s_part[16][kWtKeys];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int kvh = blockIdx.x % a.Hkv;
  const int kt = (int)(blockIdx.x / a.Hkv % key_tiles), b = (int)(blockIdx.x / a.Hkv / key_tiles);
  WeightRequest r;
  if (!weight_request_cta(a, b, r, kt == 0 && kvh == 0)) return;
  const int k0 = kt * kWtKeys, total = r.P + r.m;
  if (k0 >= total) return;
  const int32_t* bt = a.block_table + (size_t)b * a.max_blocks;
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  const int first = r.m - r.cnt, R = r.cnt * a.g;
  // the first counted token that sees the tile's first slot
  const int tok0 = max(0, k0 - r.P - first);
  float w[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  int bad = 0;
  if (tok0 < r.cnt) {
    load_tile<T, D, kWtKeys>(sk, [&](int i) -> const T* { return k0 + i < total ? key_row<T>(a, bt, kvh, k0 + i, &bad) : nullptr; });
    for (int r0 = tok0 * a.g / ROWS * ROWS; r0 < R; r0 += ROWS) {
      __syncthreads();
      load_tile<T, D, ROWS>(sq, [&](int i) -> const T* {
        if (r0 + i >= R) return nullptr;
        return static_cast<const T*>(a.q) + ((size_t)weight_q_row(a, r, first + (r0 + i) / a.g) * a.Hq + kvh * a.g + (r0 + i) % a.g) * D;
      });
      for (int i = threadIdx.x; i < ROWS && r0 + i < R; i += kWtThreads) {
        // the splits that hold some of the keys this row sees
        const int splits = min(a.splits, (r.P + first + (r0 + i) / a.g) / a.chunk + 1);
        const float2* ml = a.ws_ml + weight_ws_row(a, kvh, r.off, first) + r0 + i;
        float2 x = ml[0];
        for (int k = 1; k < splits; ++k) x = weight_join(x, ml[(size_t)k * a.T * a.Hq]);
        s_lse[i] = x.x + log2f(x.y);
      }
      __syncthreads();
      float s[RT][4];
      scores<D, RT>(sq, sk, ty, tx, s);
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const int row = r0 + RT * ty + i;
        if (row >= R) continue;
        const int seen = r.P + first + row / a.g;
        const float lse = s_lse[RT * ty + i];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (k0 + 4 * tx + j <= seen) w[j] += exp2f(s[i][j] * a.scale_log2 - lse);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) s_part[ty][4 * tx + j] = w[j];
  __syncthreads();
  for (int i = threadIdx.x; i < kWtKeys; i += kWtThreads) {
    const int s = k0 + i;
    if (s >= total) continue;
    float sum = 0.0f;
#pragma unroll
    for (int y = 0; y < 16; ++y) sum += s_part[y][i];
    const size_t at = ((size_t)b * a.Hkv + kvh) * a.stride + s;
    a.weight[at] = (a.before && s < r.P ? a.decay * a.before[at] : 0.0f) + sum;
  }
  if (bad) atomicOr(&a.status[b], SPEC_DEV_BAD_BLOCK);
}

template <typename T, int D, int RT>
static cudaError_t launch_cc(const WeightArgs& a, const WeightPlan& p, cudaStream_t stream) {
  const int dyn = 2 * D * (64 + kWtPad) * (int)sizeof(float);
  cudaError_t e = cudaFuncSetAttribute(weight_stats_cc_kernel<T, D, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize, dyn);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(weight_sums_cc_kernel<T, D, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize, dyn);
  if (e != cudaSuccess) return e;
  if (p.tiles > 0) {
    weight_stats_cc_kernel<T, D, RT><<<(unsigned)(p.tiles * a.Hkv * p.splits), kWtThreads, dyn, stream>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  const int key_tiles = (a.max_prefix + a.n_max + kWtKeys - 1) / kWtKeys;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((long long)a.B * key_tiles * a.Hkv), 1, 1);
  cfg.blockDim = dim3(kWtThreads, 1, 1);
  cfg.dynamicSmemBytes = dyn;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];  // a programmatic dependent of the statistics
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.tiles > 0 ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, weight_sums_cc_kernel<T, D, RT>, a, key_tiles);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// Rows per tile of the CUDA-core kernels: the most that a request has decides.
static int weight_cc_rows(int n_max, int window, int g) {
  return (long long)(window > 0 ? std::min(window, n_max) : n_max) * g <= kWtFewRows ? kWtFewRows : kWtRows;
}

cudaError_t launch_weight_cc(const WeightArgs& a, const WeightPlan& p, cudaStream_t stream) {
  if (weight_cc_rows(a.n_max, a.window, a.g) == kWtFewRows)
    return a.D == 64 ? launch_cc<float, 64, 1>(a, p, stream) : launch_cc<float, 128, 1>(a, p, stream);
  return a.D == 64 ? launch_cc<float, 64, 4>(a, p, stream) : launch_cc<float, 128, 4>(a, p, stream);
}

constexpr int kWtSms = 152;  // the plan's SM count (part of the workspace query)

// Row tiles of M rows, and key splits, of 512 keys at least, while the tiles alone
// are fewer than two items per SM.  Where most requests fill no tile (single
// tokens, paths) an item is at most 2048 keys: their lengths differ, and whole
// ones leave SMs idle at the end.
static WeightPlan weight_plan(int B, int T, int n_max, int max_prefix, int Hq, int Hkv, int window, int M, int* per_req) {
  const int g = Hq / Hkv;
  const long long packed = (long long)T * g / M + B;
  const long long each = ((long long)(window > 0 ? std::min(window, n_max) : n_max) * g + M - 1) / M;
  WeightPlan p = {};
  *per_req = each * B < packed ? (int)each : 0;
  p.tiles = std::min(each * B, packed);
  const long long keys = (long long)max_prefix + n_max, work = std::max(1LL, p.tiles * Hkv);
  const bool few = p.tiles < 2LL * B;
  long long chunk = work >= 2LL * kWtSms ? keys : std::max(512LL, keys * work / (2LL * kWtSms));
  if (few) chunk = std::min(chunk, 2048LL);
  p.chunk = (int)std::max(128LL, (chunk + 127) / 128 * 128);
  p.splits = (int)std::max(1LL, (keys + p.chunk - 1) / p.chunk);
  return p;
}

static spec_status weight_shape_check(int B, int T, int n_max, int max_prefix, int Hq, int Hkv, int D, int block_size) {
  if (B < 0 || T < 0 || n_max < 0 || max_prefix < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0) return SPEC_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return SPEC_ERR_UNSUPPORTED;
  if (block_size < 8 || block_size > 65536 || (block_size & (block_size - 1))) return SPEC_ERR_UNSUPPORTED;
  if (B > 65535 || Hkv > 65535 || (long long)n_max * (Hq / Hkv) >= (1LL << 30) || (long long)max_prefix + n_max >= (1LL << 30) ||
      (long long)T * Hq >= (1LL << 31))
    return SPEC_ERR_UNSUPPORTED;
  return SPEC_OK;
}

static size_t weight_ws_bytes(int splits, int T, int Hq, bool tc) {
  return (size_t)T * Hq * ((size_t)splits * (tc ? kWtParts : 1) * sizeof(float2) + (tc ? sizeof(float) : 0));
}

// Parts of a request's rows whose sums are taken apart, where the items of 256 keys
// alone do not reach every SM: for a dozen items an SM, half of which are above a
// prompt's diagonal and fall away.  One prompt of 4000 tokens with 8, 4 and 2 kv-heads
// (128, 64 and 32 items): 149, 192 and 144 us whole, 98, 67 and 32 us in 15 or 16 parts.
// An item more costs a CTA some 7 us (its keys' load, the score buffers run dry).  Whole
// calls (statistics too, 8 kv-heads, L2 flushed), whole rows, the best number of parts,
// and 12 parts: 144 items 259, 222 (3 parts), 230 us; 160 items 280, 231 (2), 247; 176
// items 323, 289 (6), 298; 208 items 395, 384 (6), 384; 240 items 477, 479 (8), 500; 256
// items 532, 558 (6), 569.  So from 152 to some 200 items two to six parts would be
// faster than the whole rows that the rule takes (up to 18 %).
static int weight_parts(int B, int n_max, int max_prefix, int Hkv) {
  const long long items = std::max(1LL, ((long long)max_prefix + n_max + 255) / 256 * B * Hkv);
  return items >= kWtSms ? 1 : (int)std::min(16LL, (12LL * kWtSms + items - 1) / items);
}
static size_t weight_parts_bytes(int parts, int B, int n_max, int max_prefix, int Hkv) {
  return parts > 1 ? (size_t)parts * B * Hkv * ((size_t)max_prefix + n_max) * sizeof(float) : 0;
}

}  // namespace spectree

using namespace spectree;

extern "C" {

// What no call of these sizes or smaller ones exceeds, whatever its window and
// type: fewer rows and keys split further, so the need itself does not grow with
// the sizes (32/8 heads, D 128, prefix 4096: 38 KB for one request of 8 rows, 21 for
// 8 requests of one).  Splits: weight_plan's chunk is at least 512 keys,
// and, but for the 2048 of few rows, the keys that 2 kWtSms items of one row tile
// have (rounded down once: one split more).  Parts: fewer than kWtSms items of 256
// keys, in at most 12 kWtSms parts of items in all and one more each.
size_t spec_weight_workspace_size(int B, int T, int n_max, int max_prefix, int Hq, int Hkv, int D) {
  if (B <= 0 || T <= 0 || n_max <= 0 || weight_shape_check(B, T, n_max, max_prefix, Hq, Hkv, D, 16) != SPEC_OK) return 256;
  const long long keys = (long long)max_prefix + n_max;
  const int splits = (int)std::max(std::min((keys + 511) / 512, 2LL * kWtSms / Hkv + 2), (keys + 2047) / 2048);
  const bool parts = (long long)n_max * (Hq / Hkv) > weight_tc_rows(Hq / Hkv);
  const long long part_sums = parts ? 16 * std::min(B * keys * Hkv, 13LL * kWtSms * 16) : 0;
  return std::max<size_t>(256, weight_ws_bytes(splits, T, Hq, true) + part_sums * sizeof(float));
}

spec_status spec_attention_weight(const void* q, const void* k_cache, const int32_t* block_table, int max_blocks,
                                  int block_size, int num_blocks, const int32_t* prefix_len, const int32_t* seq_off,
                                  const int32_t* path, int path_stride, const int32_t* accept_len, int window, int B,
                                  int T, int n_max, int max_prefix, int Hq, int Hkv, int D, spec_dtype dtype,
                                  float scale, float decay, const float* before, float* weight,
                                  long long weight_stride, void* workspace, size_t workspace_bytes, int32_t* status,
                                  void* stream) {
  SPEC_NVTX_RANGE("spec_attention_weight");
  if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_INVALID_ARG;
  if (!(scale >= 0.0f && scale < INFINITY) || !(decay >= 0.0f && decay < INFINITY)) return SPEC_ERR_INVALID_ARG;
  if (window < 0 || weight_stride < 0 || (path && path_stride <= 0) || (path == nullptr) != (accept_len == nullptr))
    return SPEC_ERR_INVALID_ARG;
  const spec_status sc = weight_shape_check(B, T, n_max, max_prefix, Hq, Hkv, D, block_size);
  if (sc != SPEC_OK) return sc;
  if (weight_stride > (1LL << 31)) return SPEC_ERR_UNSUPPORTED;
  if (B == 0) return SPEC_OK;
  if (!k_cache || !block_table || !prefix_len || !seq_off || !weight || !status || max_blocks <= 0 || num_blocks <= 0 ||
      (!q && T > 0))
    return SPEC_ERR_INVALID_ARG;
  if (((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k_cache)) & 15) != 0) return SPEC_ERR_INVALID_ARG;
  WeightArgs a = {};
  const bool tc = dtype == SPEC_BF16;
  // the tensor-core path names cache rows by 32-bit coordinates
  if (tc && (long long)num_blocks * Hkv * block_size >= (long long)INT32_MAX) return SPEC_ERR_UNSUPPORTED;
  const WeightPlan plan = weight_plan(B, T, n_max, max_prefix, Hq, Hkv, window, tc ? weight_tc_rows(Hq / Hkv) : weight_cc_rows(n_max, window, Hq / Hkv), &a.per_req);
  const long long key_tiles = ((long long)max_prefix + n_max + kWtKeys - 1) / kWtKeys;
  if (plan.tiles * Hkv * plan.splits > (long long)INT32_MAX / 2 || key_tiles * B * Hkv > (long long)INT32_MAX / 2) return SPEC_ERR_UNSUPPORTED;
  if (key_tiles == 0) return SPEC_OK;
  // only requests of more rows than one item's take them in parts
  const long long rows = (long long)(window > 0 ? std::min(window, n_max) : n_max) * (Hq / Hkv);
  const bool rowless = T == 0 || n_max == 0;  // no request can have a row: nothing goes through the workspace
  a.parts = tc && !rowless && rows > weight_tc_rows(Hq / Hkv) ? weight_parts(B, n_max, max_prefix, Hkv) : 1;
  const size_t sums = rowless ? 0 : weight_ws_bytes(plan.splits, T, Hq, tc), need = sums + weight_parts_bytes(a.parts, B, n_max, max_prefix, Hkv);
  if (need > 0 && (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 15))) return SPEC_ERR_WORKSPACE;
  a.q = q;
  a.k_cache = k_cache;
  a.block_table = block_table;
  a.prefix_len = prefix_len;
  a.seq_off = seq_off;
  a.path = path;
  a.accept_len = accept_len;
  a.before = before;
  a.weight = weight;
  a.status = status;
  a.ws_ml = static_cast<float2*>(workspace);
  if (a.parts > 1) a.ws_part = reinterpret_cast<float*>(static_cast<char*>(workspace) + sums);
  if (tc && sums > 0) a.ws_lse = static_cast<float*>(workspace) + (size_t)plan.splits * T * Hq * kWtParts * 2;
  a.stride = weight_stride;
  a.path_stride = path_stride;
  a.window = window;
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
  // The tensor-core kernels hide a key by -inf before the scaling, and -inf * 0 is
  // NaN: the smallest float stands for a scale of 0.
  a.scale_log2 = std::max(scale * 1.4426950408889634f, 0x1p-149f);
  a.decay = decay;
  cudaStream_t st = (cudaStream_t)stream;
  if (need > 0) spec_workspace_canary(workspace, need, st);
  return (tc ? launch_weight_tc(a, st) : launch_weight_cc(a, plan, st)) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // extern "C"
