// Eviction from the paged K/V cache by weight: each layer and kv-head of a row
// keeps its first slots, its last ones and, of the others, the heaviest, and
// what is kept is copied in slot order to another row of the block table.
//
// Out of place: the row's pages may be shared (a fork's full pages are), and a
// copy needs no order among the moves.  The old row's pages go back by
// spec_pages_free, or stay (the whole cache for the target, the short one for a
// draft).
//
// Two kernels.  The selection (a CTA for each layer, row and kv-head) finds the
// border weight by histograms, 2048 equal bins between the least and the largest
// key that compete (an order-preserving whole number), then 2048 within the bin
// that holds the border, and so on; then it lists the kept slots in one ordered
// pass; equal weights at the border are taken from the lowest slot.  Rows of up
// to 16384 slots (49152 where SMs are idle) are read once and their keys kept in
// shared memory.  The copy moves the listed rows, 16 bytes a lane; with rows
// enough for every SM, or few enough for one CTA, the CTA that selected them moves
// them, while others select.
// Measured: four rows of 6000 to 8192 slots cut to 1024 in 32 layers 233 us (1.1
// GB, 4.8 TB/s; 239 with a kernel of its own for the copy, of which the selection
// took 63); 64 rows of up to 1024 to 256 in two layers 59 us (65).  What is lost
// to HBM's 6.8 TB/s is a CTA's own chain: some 16 us from its row to its list.
#include <algorithm>

#include "common.cuh"

namespace spectree {

constexpr int kSelThreads = 512, kSelShort = 128;  // per row, and per row of a table of up to kSelShortSlots
constexpr int kSelShortSlots = 2048;
constexpr int kSelBins = 2048;
constexpr int kSelRun = 4;          // neighbouring slots per thread of the listing
constexpr int kSelHeld = 16384;     // most keys held in shared memory (three CTAs an SM), and
constexpr int kSelHeldOne = 49152;  // where there is at most one CTA for an SM
constexpr int kGatherThreads = 256;
constexpr int kGatherCtas = 8;      // per SM
constexpr int kGatherVec = 4;       // 16-byte vectors of K and V per thread and step

struct EvictArgs {
  char* const* k_caches;
  char* const* v_caches;
  const int32_t* table;
  const int32_t* src;
  const int32_t* dst;
  const int32_t* len;
  const int32_t* keep;
  float* weight;
  int32_t* slots;
  int32_t* new_len;
  int32_t* status;
  long long stride;                 // weights of one (layer, row, kv-head)
  int layers, B, max_blocks, bs_log2, num_blocks, N, keep_max, first, last, Hkv;
  int vec;                          // 16-byte vectors of a row
  int held;                         // keys that the selection's shared memory holds
};

// A key whose order as a whole number is the weights': NaN lowest, -0 as +0.
__device__ __forceinline__ uint32_t weight_key(float x) {
  if (x != x) return 0;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// The weight of a key, but for what a key does not tell apart (NaNs, the zeros) or
// does not know (a slot that stays whatever it weighs).
__device__ __forceinline__ bool key_weight(uint32_t k, float& x) {
  x = __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
  return k != 0u && k != 0x80000000u && k != ~0u;
}

// What row i of the call keeps, or the SPEC_DEV_* bits that stop it, its pages
// apart (the same in every thread of every CTA).
struct EvictRow {
  int src, dst, len, kept, first, last, bad;
};
template <int kThreads>
__device__ __forceinline__ EvictRow evict_row(const EvictArgs& a, int i) {
  EvictRow r = {a.src[i], a.dst[i], a.len[i], 0, 0, 0, 0};
  const int keep = a.keep ? a.keep[i] : a.keep_max;
  int other = 0;
  for (int j = threadIdx.x; j < a.N; j += kThreads) other |= (j != i && a.dst[j] == r.dst) || a.src[j] == r.dst;
  other = __syncthreads_or(other);
  if (other || r.src < 0 || r.src >= a.B || r.dst < 0 || r.dst >= a.B || r.src == r.dst || r.len < 0 || keep < 0 || keep > a.keep_max) {
    r.bad = SPEC_DEV_BAD_ROW;
    return r;
  }
  r.kept = min(keep, r.len);
  r.first = min(a.first, r.kept);
  r.last = min(a.last, r.kept - r.first);
  if (r.len > (1 << 30) || r.len > (long long)a.max_blocks << a.bs_log2 || (a.weight && r.len > a.stride)) r.bad = SPEC_DEV_CAPACITY;
  return r;
}

// Kept rows j0 .. of (layer, row i, kv-head h), K and V: as many as the CTA's
// threads hold kGatherVec vectors each.
template <int kThreads>
__device__ __forceinline__ void copy_rows(const EvictArgs& a, int layer, int i, int h, const int32_t* slots, int j0, int kept) {
  const int32_t *from = a.table + (size_t)a.src[i] * a.max_blocks, *to = a.table + (size_t)a.dst[i] * a.max_blocks;
  uint4 *kc = reinterpret_cast<uint4*>(a.k_caches[layer]), *vc = reinterpret_cast<uint4*>(a.v_caches[layer]);
  const int within = (1 << a.bs_log2) - 1;
  uint4 k[kGatherVec], v[kGatherVec];
  long long put[kGatherVec];
#pragma unroll
  for (int e = 0; e < kGatherVec; ++e) {
    const int x = threadIdx.x + e * kThreads, j = j0 + x / a.vec, c = x % a.vec;
    put[e] = -1;
    if (j < kept) {
      const int s = slots[j];
      const long long get = ((((long long)from[s >> a.bs_log2] * a.Hkv + h) << a.bs_log2) + (s & within)) * a.vec + c;
      put[e] = ((((long long)to[j >> a.bs_log2] * a.Hkv + h) << a.bs_log2) + (j & within)) * a.vec + c;
      k[e] = kc[get];
      v[e] = vc[get];
    }
  }
#pragma unroll
  for (int e = 0; e < kGatherVec; ++e)
    if (put[e] >= 0) {
      kc[put[e]] = k[e];
      vc[put[e]] = v[e];
    }
}

// COPY: the CTA moves its rows itself.
template <int kThreads, bool COPY>
__global__ void __launch_bounds__(kThreads) evict_select_kernel(const EvictArgs a) {
  constexpr int kWarps = kThreads / 32;
  extern __shared__ uint32_t keys[];  // of the row's slots
  __shared__ uint32_t hist[kSelBins];
  __shared__ uint32_t s_warp[kWarps];
  __shared__ uint32_t s_bin, s_left, s_least, s_most;
  // the copy's kernel may launch early; a call's last kernel lets none, since tree
  // attention reads cache rows before it waits for the kernel before it
  if (!COPY) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int h = blockIdx.x % a.Hkv, i = blockIdx.x / a.Hkv % a.N, layer = blockIdx.x / a.Hkv / a.N;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  EvictRow r = evict_row<kThreads>(a, i);
  const bool cached = r.len <= a.held;
  const float* w = nullptr;
  // the slots outside [begin, end) stay whatever they weigh: their key is the
  // largest, which no weight has
  const int begin = r.first, end = r.len - r.last;
  auto key_of = [&](int s, float x) -> uint32_t { return s < begin || s >= end ? ~0u : weight_key(x); };
  if (!r.bad) {
    // the weights (sixteen loads at a time) and both rows' pages in one go
    if (a.weight) w = a.weight + (((size_t)layer * a.B + r.src) * a.Hkv + h) * a.stride;
    if (cached) {
      for (int s0 = t; s0 < r.len; s0 += 16 * kThreads) {
        float x[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = w && s0 + e * kThreads < r.len ? w[s0 + e * kThreads] : 0.0f;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int s = s0 + e * kThreads;
          if (s < r.len) keys[s] = key_of(s, x[e]);
        }
      }
    }
    const int32_t *from = a.table + (size_t)r.src * a.max_blocks, *into = a.table + (size_t)r.dst * a.max_blocks;
    const long long bs = 1LL << a.bs_log2;
    const int pages = (int)((r.len + bs - 1) >> a.bs_log2), need = (int)((r.kept + bs - 1) >> a.bs_log2);
    int bb = 0;
    for (int j = t; j < pages; j += kThreads) bb |= from[j] < 0 || from[j] >= a.num_blocks;
    for (int j = t; j < need; j += kThreads) bb |= into[j] < 0 || into[j] >= a.num_blocks;
    if (t == 0) {
      s_least = ~0u;
      s_most = 0;
    }
    if (__syncthreads_or(bb)) r.bad = SPEC_DEV_BAD_BLOCK;
  }
  int32_t* out = a.slots + (((size_t)layer * a.N + i) * a.Hkv + h) * a.keep_max;
  if (layer == 0 && h == 0 && t == 0) {
    a.status[i] = r.bad;
    a.new_len[i] = r.bad ? 0 : r.kept;
  }
  const int kept = r.bad ? 0 : r.kept;
  for (int j = kept + t; j < a.keep_max; j += kThreads) out[j] = -1;
  if (kept == 0) return;
  float* to = a.weight ? a.weight + (((size_t)layer * a.B + r.dst) * a.Hkv + h) * a.stride : nullptr;
  const bool all = kept == r.len;

  // border: every key above it stays, and the first `ties` of those equal to it.
  // Of the competing keys within [low, low + 2^width) a histogram of 2048 equal bins
  // tells the one that holds the border; the next round's range is that bin.
  uint32_t border = 0, ties = 0;
  if (!all) {
    auto key_at = [&](int s) -> uint32_t { return cached ? keys[s] : w ? weight_key(w[s]) : weight_key(0.0f); };
    uint32_t least = ~0u, most = 0;
    for (int s = begin + t; s < end; s += kThreads) {
      const uint32_t k = key_at(s);
      least = min(least, k);
      most = max(most, k);
    }
    least = __reduce_min_sync(0xffffffffu, least);
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) {
      atomicMin(&s_least, least);
      atomicMax(&s_most, most);
    }
    __syncthreads();
    uint32_t low = s_least, high = s_most;
    ties = kept - r.first - r.last;  // 0: the ends alone stay, and no key is above `most`
    if (ties == 0) border = high;
    for (int shift = max(0, 21 - __clz(high - low)); ties > 0;) {
      for (int j = t; j < kSelBins; j += kThreads) hist[j] = 0;
      __syncthreads();
#pragma unroll 4
      for (int s = begin + t; s < end; s += kThreads) {
        const uint32_t k = key_at(s);
        if (k >= low && k <= high) atomicAdd(&hist[(k - low) >> shift], 1u);
      }
      __syncthreads();
      // the bin where the count from the top reaches `ties`: each thread holds kBins
      // bins in a row, counted from the top
      constexpr int kBins = kSelBins / kThreads;
      uint32_t c[kBins], sum = 0;
#pragma unroll
      for (int e = 0; e < kBins; ++e) sum += c[e] = hist[kSelBins - 1 - (kBins * t + e)];
      uint32_t at = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, at, o);
        if (lane >= o) at += y;
      }
      if (lane == 31) s_warp[warp] = at;
      __syncthreads();
      at -= sum;
      for (int k = 0; k < warp; ++k) at += s_warp[k];
#pragma unroll
      for (int e = 0; e < kBins; ++e) {
        if (at < ties && ties <= at + c[e]) {
          s_bin = kSelBins - 1 - (kBins * t + e);
          s_left = ties - at;
        }
        at += c[e];
      }
      __syncthreads();
      low += s_bin << shift;
      ties = s_left;
      border = low;
      if (shift == 0) break;
      high = low + ((1u << shift) - 1);
      shift = max(0, shift - 11);
    }
  }

  // the kept slots in order, kSelRun neighbours to a thread: counts of larger and
  // of equal keys (the first `ties` of these stay) go through one scan
  uint32_t big = 0, equal = 0;  // of the slots before this round
  for (int s0 = 0; s0 < r.len; s0 += kThreads * kSelRun) {
    const int s = s0 + t * kSelRun;
    uint32_t g = 0, q = 0;  // bit e: slot s + e
    uint32_t key[kSelRun];
#pragma unroll
    for (int e = 0; e < kSelRun; ++e) {
      if (s + e >= r.len) continue;
      const uint32_t k = key[e] = cached ? keys[s + e] : key_of(s + e, w ? w[s + e] : 0.0f);
      g |= (uint32_t)(all || k > border) << e;
      q |= (uint32_t)(!all && k == border) << e;
    }
    const uint32_t mine = __popc(g) | (uint32_t)__popc(q) << 16;
    uint32_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    __syncthreads();  // s_warp of the round before has been read
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    uint32_t before = incl - mine, total = 0;  // 16 bits each: at most 2048 of a round
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      const uint32_t y = s_warp[k];
      before += k < warp ? y : 0;
      total += y;
    }
    uint32_t bg = big + (before & 0xffffu), bq = equal + (before >> 16);
#pragma unroll
    for (int e = 0; e < kSelRun; ++e) {
      const bool heavy = g >> e & 1, even = q >> e & 1;
      if (heavy || (even && bq < ties)) {
        const uint32_t at = bg + min(bq, ties);
        out[at] = s + e;
        if (to) {
          float x;
          to[at] = key_weight(key[e], x) ? x : w[s + e];
        }
      }
      bg += heavy;
      bq += even;
    }
    big += total & 0xffffu;
    equal += total >> 16;
  }
  if (COPY) {
    __syncthreads();  // the list is whole
    const int rows = kThreads * kGatherVec / a.vec;
    for (int j0 = 0; j0 < kept; j0 += rows) copy_rows<kThreads>(a, layer, i, h, out, j0, kept);
  }
}

__global__ void __launch_bounds__(kGatherThreads) evict_gather_kernel(const EvictArgs a, long long units, int per_head) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int rows = kGatherThreads * kGatherVec / a.vec;  // of a unit
  for (long long unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int part = (int)(unit % per_head);
    const long long head = unit / per_head;
    const int h = (int)(head % a.Hkv), i = (int)(head / a.Hkv % a.N), layer = (int)(head / a.Hkv / a.N);
    const int kept = a.new_len[i];
    if (part * rows < kept) copy_rows<kGatherThreads>(a, layer, i, h, a.slots + (size_t)head * a.keep_max, part * rows, kept);
  }
}

}  // namespace spectree

using namespace spectree;

extern "C" spec_status spec_kv_evict(void* const* k_caches, void* const* v_caches, int layers, const int32_t* block_table,
                                     int B, int max_blocks, int block_size, int num_blocks, const int32_t* src,
                                     const int32_t* dst, const int32_t* len, const int32_t* keep, int N, int keep_max,
                                     int first, int last, float* weight, long long weight_stride, int Hkv, int D,
                                     spec_dtype dtype, int32_t* slots, int32_t* new_len, int32_t* status, void* stream) {
  SPEC_NVTX_RANGE("spec_kv_evict");
  if (layers <= 0 || B < 0 || max_blocks <= 0 || num_blocks <= 0 || N < 0 || keep_max < 0 || first < 0 || last < 0 ||
      Hkv <= 0 || weight_stride < 0)
    return SPEC_ERR_INVALID_ARG;
  if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return SPEC_ERR_UNSUPPORTED;
  if (block_size < 8 || block_size > 65536 || (block_size & (block_size - 1))) return SPEC_ERR_UNSUPPORTED;
  const long long heads = (long long)layers * N * Hkv;
  if (Hkv > 65535 || layers > 32767 || N > 65535 || heads > INT32_MAX || keep_max > (1 << 30) ||
      weight_stride > (1LL << 31) || (long long)B * max_blocks > (1LL << 40))
    return SPEC_ERR_UNSUPPORTED;
  if (N == 0) return SPEC_OK;
  if (!k_caches || !v_caches || !block_table || !src || !dst || !len || !new_len || !status || (keep_max > 0 && !slots))
    return SPEC_ERR_INVALID_ARG;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return SPEC_ERR_CUDA;
  EvictArgs a = {};
  a.k_caches = (char* const*)k_caches;
  a.v_caches = (char* const*)v_caches;
  a.table = block_table;
  a.src = src;
  a.dst = dst;
  a.len = len;
  a.keep = keep;
  a.weight = weight;
  a.slots = slots;
  a.new_len = new_len;
  a.status = status;
  a.stride = weight_stride;
  a.layers = layers;
  a.B = B;
  a.max_blocks = max_blocks;
  while ((1 << a.bs_log2) < block_size) ++a.bs_log2;
  a.num_blocks = num_blocks;
  a.N = N;
  a.keep_max = keep_max;
  a.first = first;
  a.last = last;
  a.Hkv = Hkv;
  a.vec = D * (dtype == SPEC_F32 ? 4 : 2) / 16;
  cudaStream_t st = (cudaStream_t)stream;
  // room for the keys of the longest row that the table and the weights allow
  const long long most = std::min((long long)max_blocks << a.bs_log2, weight ? weight_stride : (1LL << 30));
  a.held = (int)std::min<long long>(most, heads <= sms ? kSelHeldOne : kSelHeld);
  const int dyn = a.held * (int)sizeof(uint32_t);
  const bool small = most <= kSelShortSlots;
  // With rows enough for every SM a CTA moves what it has selected while others
  // select; with fewer, the copy is a kernel of its own that every SM takes part in,
  // unless it is so short that the launch would cost more.
  const bool copy = heads >= 2LL * sms || (long long)keep_max * a.vec <= 8LL * (small ? kSelShort : kSelThreads) * kGatherVec;
  const auto select = small ? (copy ? evict_select_kernel<kSelShort, true> : evict_select_kernel<kSelShort, false>)
                            : (copy ? evict_select_kernel<kSelThreads, true> : evict_select_kernel<kSelThreads, false>);
  // the limit belongs to the function, not to this call: one value for every call, as
  // another thread's may set it between this one's set and its launch
  constexpr int kDynMax = kSelHeldOne * (int)sizeof(uint32_t);
  if (dyn > 32 * 1024 && cudaFuncSetAttribute(select, cudaFuncAttributeMaxDynamicSharedMemorySize, kDynMax) != cudaSuccess) return SPEC_ERR_CUDA;
  select<<<(unsigned)heads, small ? kSelShort : kSelThreads, dyn, st>>>(a);
  SPEC_LAUNCH_CHECK();
  if (keep_max == 0 || copy) return SPEC_OK;
  const int rows = kGatherThreads * kGatherVec / a.vec, per_head = (keep_max + rows - 1) / rows;
  const long long units = heads * per_head;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min<long long>(units, (long long)kGatherCtas * sms), 1, 1);
  cfg.blockDim = dim3(kGatherThreads, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, evict_gather_kernel, a, units, per_head);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}
