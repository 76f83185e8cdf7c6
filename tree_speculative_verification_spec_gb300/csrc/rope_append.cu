// Head norms, rotary positions and the append, in one pass over a projection's
// output: a token's row holds Hq query, Hkv key and Hkv value heads; queries
// and keys are normalised (x w / sqrt(mean x^2 + eps)) and rotated, keys and
// values go to their paged slots, queries to q_out.
//
// Angles.  Pair i of a head turns by t = position * inv_freq[i] radians.  At
// position 10^6 an fp32 product is off by 0.03 radians, so the turn is taken in
// 64 bits, t / 2pi less its nearest whole number (an error of 2^-52 of the
// turns), and what is left, at most half a turn, goes to fp32 and sincospi: an
// error of 2^-24 of the angle left.  A CTA computes the table of its tokens
// once, for every head.
//
// Layout.  A head row is read by LPH = D / (2 VE) lanes of two 16-byte vectors
// each (VE elements a vector).  Lane c's vectors are the two halves of the same
// pairs, so that a rotation needs no other lane.
//
// What bounds it, and what it measured (one GB300): HBM and the issue slots (62 %
// used; 100 us for a prompt of 16384 tokens, 32/8 heads, D 128, bf16, before the
// arithmetic was paired, 81 before the tables lost their bank conflicts).  That
// prompt 77 us, 5.2 TB/s; four prompts of 1500 to 2048 tokens with 64/8 heads and
// three axes 57 us; trees of 64 requests 19 us, of which a CTA's own chain (packing,
// table, rows, angles) is most; a few tokens 5 us on the GPU.
#include <algorithm>

#include "common.cuh"

namespace spectree {

constexpr int kRopeThreads = 256;
constexpr int kRopeTokens = 4;              // most tokens per CTA
constexpr int kRopeMaxPos = 1 << 24;        // positions
enum RopeMode { kRopeHalves = 0, kRopeNeighbours = 1, kRopeShared = 2 };

struct RopeArgs {
  const char* qkv;
  long long row_bytes;                      // from one token's row to the next
  const void* q_norm;
  const void* k_norm;
  const float* inv_freq;
  const int32_t* axis;
  const int32_t* pos_base;
  const int32_t* pos;
  char* q_out;
  char* k_cache;
  char* v_cache;
  const int32_t* block_table;
  const int32_t* prefix_len;
  const int32_t* tree_off;
  int32_t* status;
  float eps;
  int rot, axes, mode;
  int max_blocks, bs_log2, num_blocks, B, T, n_max, Hq, Hkv;
};

// One 16-byte vector as pairs of fp32 values, and back (rounded to nearest).
template <typename T> struct Vec;
template <> struct Vec<float> {
  static constexpr int N = 4;
  __device__ static void open(const uint4& u, float2* x) {
    x[0] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
    x[1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
  }
  __device__ static uint4 close(const float2* x) {
    return make_uint4(__float_as_uint(x[0].x), __float_as_uint(x[0].y), __float_as_uint(x[1].x), __float_as_uint(x[1].y));
  }
};
template <> struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  __device__ static void open(const uint4& u, float2* x) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
  __device__ static uint4 close(const float2* x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __float22bfloat162_rn(x[i]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// The SPEC_DEV_* bits of a request's own arguments.
__device__ __forceinline__ int rope_check(const RopeArgs& a, int off, int n, int P) {
  if (off < 0 || n < 0 || n > a.n_max || n > a.T - off) return SPEC_DEV_BAD_TREE;
  const long long end = (long long)P + n;
  return P < 0 || end > ((long long)a.max_blocks << a.bs_log2) || end > INT32_MAX ? SPEC_DEV_CAPACITY : 0;
}

// Token tiles of `tt` tokens are numbered from floor(tree_off[b] / tt) + b: at
// least ceil(n_b / tt) of them lie before the next request's first, and
// floor(T / tt) + B cover every batch of T tokens without a prefix sum.
template <typename T, int D, int MODE>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_append_kernel(const RopeArgs a, int tt) {
  constexpr int VE = Vec<T>::N, LPH = D / (2 * VE), GROUPS = kRopeThreads / LPH, U = 2;
  __shared__ __align__(16) float s_cos[kRopeTokens][D / 2], s_sin[kRopeTokens][D / 2], s_norm[2][D];
  __shared__ float s_row[MODE == kRopeShared ? GROUPS : 1][D];  // a normalised row (pairs that cross lanes)
  __shared__ long long s_slot[kRopeTokens];  // row of the token's slot in kv-head 0 of its page
  __shared__ int s_bad[kRopeTokens];
  // The tables lie so that lanes that read 16 bytes each, of neighbouring vectors,
  // read neighbouring 16 bytes: element j of vector v at ((j / 4) n + v) 4 + j % 4,
  // n vectors in all (32 bytes apart, eight lanes' reads fell on four banks twice).
  constexpr int PV = MODE == kRopeHalves ? VE : 4;  // pairs per vector of the angles' table
  auto pair_at = [](int pair) { return ((pair % PV / 4) * (D / 2 / PV) + pair / PV) * 4 + pair % 4; };
  auto norm_at = [](int el) { return ((el % VE / 4) * (D / VE) + el / VE) * 4 + el % 4; };
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tile = blockIdx.x, t = threadIdx.x;
  if (t < kRopeTokens) s_bad[t] = 0;
  // the last request whose first tile is not above this one
  int count = 0;
  for (int j0 = 0; j0 < a.B; j0 += kRopeThreads) {
    const int j = j0 + t;
    count += __syncthreads_count(j < a.B && a.tree_off[j] / tt + j <= tile);
  }
  const int b = max(count - 1, 0);
  const int off = a.tree_off[b], n = a.tree_off[b + 1] - off, P = a.prefix_len[b];
  // CTA 0 flags every request whose arguments are out of range
  if (tile == 0) {
    for (int j = t; j < a.B; j += kRopeThreads) {
      const int o = a.tree_off[j];
      const int bad = rope_check(a, o, a.tree_off[j + 1] - o, a.prefix_len[j]);
      if (bad) atomicOr(&a.status[j], bad);
    }
  }
  if (n == 0 || rope_check(a, off, n, P)) return;
  const long long at = (long long)tile - (off / tt + b);
  if (at < 0 || at * tt >= n) return;
  const int u0 = (int)at * tt, nt = min(tt, n - u0);
  const int32_t* bt = a.block_table + (size_t)b * a.max_blocks;

  const int heads = a.Hq + 2 * a.Hkv;
  const int group = t / LPH, c = t % LPH;
  // lane c's vectors: the rotated ones by pairs of halves, the others by two
  const int rv = MODE == kRopeHalves ? a.rot / (2 * VE) : 0, half = D / (2 * VE);
  const int va = c < rv ? c : rv + c, vb = c < rv ? c + rv : half + c;
  const char* rows = a.qkv + (long long)(off + u0) * a.row_bytes;
  uint4 lo[U] = {}, hi[U] = {};
  int k = 0, h = group;  // this group's next (token, head), GROUPS heads on
  auto load = [&]() {
    int kk = k, hh = h;
#pragma unroll
    for (int e = 0; e < U; ++e, hh += GROUPS) {
      while (hh >= heads) hh -= heads, ++kk;
      if (kk < nt) {
        const char* row = rows + (long long)kk * a.row_bytes + (size_t)hh * (D * sizeof(T));
        lo[e] = *reinterpret_cast<const uint4*>(row + va * 16);
        hi[e] = *reinterpret_cast<const uint4*>(row + vb * 16);
      }
    }
  };
  load();
  // a bad page leaves the whole request untouched, so every CTA looks at all of them
  int bb = 0;
  for (int pg = (P >> a.bs_log2) + t; pg <= (P + n - 1) >> a.bs_log2; pg += kRopeThreads) bb |= bt[pg] < 0 || bt[pg] >= a.num_blocks;
  if (t < nt) {
    const int s = P + u0 + t;
    s_slot[t] = (((long long)bt[s >> a.bs_log2] * a.Hkv) << a.bs_log2) + (s & ((1 << a.bs_log2) - 1));
  }
  for (int i = t; i < 2 * D; i += kRopeThreads) {
    const T* norm = static_cast<const T*>(i < D ? a.q_norm : a.k_norm);
    if (norm) s_norm[i / D][norm_at(i % D)] = to_f32(norm[i % D]);
  }
  // the tokens' angles
  const int np = a.rot / 2;
  const int base = a.pos_base ? a.pos_base[b] : P;
  for (int i = t; i < nt * np; i += kRopeThreads) {
    const int j = i / np, pair = i - j * np;
    const int ax = a.axis ? a.axis[pair] : 0;
    bool ok = ax >= 0 && ax < a.axes;
    long long p = base;
    if (ok) p += a.pos ? a.pos[(size_t)ax * a.T + off + u0 + j] : u0 + j;
    ok = ok && p >= 0 && p < kRopeMaxPos;
    if (!ok) {
      s_bad[j] = 1;
      continue;
    }
    const double turns = (double)p * ((double)a.inv_freq[pair] * 0.15915494309189535);  // 1 / 2pi
    float sn, cs;
    sincospif(2.0f * (float)(turns - rint(turns)), &sn, &cs);
    s_cos[j][pair_at(pair)] = cs;
    s_sin[j][pair_at(pair)] = sn;
  }
  bb = __syncthreads_or(bb);
  if (t == 0) {
    int bad = bb ? SPEC_DEV_BAD_BLOCK : 0;
    for (int j = 0; j < nt; ++j) bad |= s_bad[j] ? SPEC_DEV_BAD_POSITION : 0;
    if (bad) atomicOr(&a.status[b], bad);
  }
  if (bb) return;

  const bool norms = a.q_norm || a.k_norm;
  for (int done = 0; done < nt * heads; done += U * GROUPS) {
    if (done > 0) load();
#pragma unroll
    for (int e = 0; e < U; ++e, h += GROUPS) {
      while (h >= heads) h -= heads, ++k;
      const bool there = k < nt;  // shuffles below: every lane of the warp comes along
      const bool is_q = h < a.Hq, is_v = h >= a.Hq + a.Hkv;
      const bool turn = there && !is_v;
      if (__any_sync(0xffffffffu, turn)) {
        float2 x[VE];  // the first vector's pairs, then the second's
        Vec<T>::open(lo[e], x);
        Vec<T>::open(hi[e], x + VE / 2);
        if (norms) {
          float2 s2 = make_float2(0.0f, 0.0f);
#pragma unroll
          for (int i = 0; i < VE; ++i) s2 = __ffma2_rn(x[i], x[i], s2);
          float ss = s2.x + s2.y;
#pragma unroll
          for (int o = LPH / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          if (turn && (is_q ? a.q_norm : a.k_norm)) {
            const float r = rsqrtf(ss * (1.0f / D) + a.eps);
            const float2 r2 = make_float2(r, r);
            const float* w = s_norm[is_q ? 0 : 1];
#pragma unroll
            for (int i = 0; i < VE; i += 2) {
              const float4 w4 = *reinterpret_cast<const float4*>(w + norm_at(i < VE / 2 ? va * VE + 2 * i : vb * VE + 2 * i - VE));
              x[i] = __fmul2_rn(__fmul2_rn(x[i], r2), make_float2(w4.x, w4.y));
              x[i + 1] = __fmul2_rn(__fmul2_rn(x[i + 1], r2), make_float2(w4.z, w4.w));
            }
          }
        }
        if (turn) {
          if (MODE == kRopeHalves) {
            if (c < rv) {
#pragma unroll
              for (int i = 0; i < VE / 2; i += 2) {
                const int at = pair_at(c * VE + 2 * i);
                const float4 c4 = *reinterpret_cast<const float4*>(&s_cos[k][at]), n4 = *reinterpret_cast<const float4*>(&s_sin[k][at]);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                  const float2 cs = j ? make_float2(c4.z, c4.w) : make_float2(c4.x, c4.y), sn = j ? make_float2(n4.z, n4.w) : make_float2(n4.x, n4.y);
                  const float2 y = x[i + j], z = x[VE / 2 + i + j];
                  x[i + j] = __ffma2_rn(y, cs, __fmul2_rn(z, make_float2(-sn.x, -sn.y)));
                  x[VE / 2 + i + j] = __ffma2_rn(z, cs, __fmul2_rn(y, sn));
                }
              }
            }
          } else if (MODE == kRopeNeighbours) {
#pragma unroll
            for (int i = 0; i < VE; ++i) {
              const int pair = i < VE / 2 ? va * (VE / 2) + i : vb * (VE / 2) + i - VE / 2;
              if (pair < np) {
                const float cs = s_cos[k][pair], sn = s_sin[k][pair];
                x[i] = make_float2(x[i].x * cs - x[i].y * sn, x[i].y * cs + x[i].x * sn);
              }
            }
          }
        }
        if (MODE == kRopeShared) {  // halves whose length is no multiple of a vector: through shared memory
          float* row = s_row[group];
#pragma unroll
          for (int i = 0; i < VE; ++i) {
            const int el = i < VE / 2 ? va * VE + 2 * i : vb * VE + 2 * i - VE;
            row[el] = x[i].x;
            row[el + 1] = x[i].y;
          }
          __syncwarp();
          auto turned = [&](int el, float v) {
            if (!there || el >= 2 * np) return v;
            return el < np ? row[el] * s_cos[k][el] - row[el + np] * s_sin[k][el] : row[el] * s_cos[k][el - np] + row[el - np] * s_sin[k][el - np];
          };
#pragma unroll
          for (int i = 0; i < VE; ++i) {
            const int el = i < VE / 2 ? va * VE + 2 * i : vb * VE + 2 * i - VE;
            x[i] = make_float2(turned(el, x[i].x), turned(el + 1, x[i].y));
          }
          __syncwarp();
        }
        if (turn) {
          lo[e] = Vec<T>::close(x);
          hi[e] = Vec<T>::close(x + VE / 2);
        }
      }
      if (there && !s_bad[k]) {
        char* dst;
        if (is_q) {
          dst = a.q_out + ((size_t)(off + u0 + k) * a.Hq + h) * (D * sizeof(T));
        } else {
          const int hk = h - a.Hq - (is_v ? a.Hkv : 0);
          dst = (is_v ? a.v_cache : a.k_cache) + (s_slot[k] + ((long long)hk << a.bs_log2)) * (D * (long long)sizeof(T));
        }
        *reinterpret_cast<uint4*>(dst + va * 16) = lo[e];
        *reinterpret_cast<uint4*>(dst + vb * 16) = hi[e];
      }
    }
  }
}

template <typename T, int D>
static cudaError_t launch_rope(const RopeArgs& a, int sms, cudaStream_t stream) {
  // Tokens per CTA: one while a CTA for each leaves room on the GPU, else four,
  // whose angles and request are looked up together (prompt of 16384: 94, 93, 84,
  // 89, 88 and 88 us with 2, 3, 4, 5, 6 and 8).
  const int tt = a.T <= 8 * sms ? 1 : kRopeTokens;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.T / tt + a.B), 1, 1);
  cfg.blockDim = dim3(kRopeThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = a.mode == kRopeHalves       ? cudaLaunchKernelEx(&cfg, rope_append_kernel<T, D, kRopeHalves>, a, tt)
                        : a.mode == kRopeNeighbours ? cudaLaunchKernelEx(&cfg, rope_append_kernel<T, D, kRopeNeighbours>, a, tt)
                                                    : cudaLaunchKernelEx(&cfg, rope_append_kernel<T, D, kRopeShared>, a, tt);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace spectree

using namespace spectree;

extern "C" spec_status spec_rope_append(const void* qkv, long long row_stride, const void* q_norm, const void* k_norm,
                                        float eps, const float* inv_freq, const int32_t* axis, int rot_dim,
                                        int pairing, const int32_t* pos_base, const int32_t* pos, int axes, void* q_out,
                                        void* k_cache, void* v_cache, const int32_t* block_table, int max_blocks,
                                        int block_size, int num_blocks, const int32_t* prefix_len,
                                        const int32_t* tree_off, int B, int T, int n_max, int Hq, int Hkv, int D,
                                        spec_dtype dtype, int32_t* status, void* stream) {
  SPEC_NVTX_RANGE("spec_rope_append");
  if (B < 0 || T < 0 || n_max < 0 || Hq <= 0 || Hkv <= 0 || max_blocks <= 0 || num_blocks <= 0) return SPEC_ERR_INVALID_ARG;
  if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return SPEC_ERR_UNSUPPORTED;
  if (block_size < 8 || block_size > 65536 || (block_size & (block_size - 1))) return SPEC_ERR_UNSUPPORTED;
  if (rot_dim < 0 || rot_dim > D || rot_dim % 2 != 0) return SPEC_ERR_INVALID_ARG;
  if (pairing != SPEC_ROPE_HALVES && pairing != SPEC_ROPE_NEIGHBOURS) return SPEC_ERR_INVALID_ARG;
  if (axes < 1 || axes > 4 || (axes > 1 && (!pos || !axis))) return SPEC_ERR_INVALID_ARG;
  if (!(eps >= 0.0f && eps < INFINITY)) return SPEC_ERR_INVALID_ARG;
  if (B > 65535 || Hq > 65535 || Hkv > 65535 || T >= (1 << 30)) return SPEC_ERR_UNSUPPORTED;
  const int size = dtype == SPEC_F32 ? 4 : 2;
  if (row_stride < (long long)(Hq + 2 * Hkv) * D || row_stride > (1LL << 40) || row_stride * size % 16 != 0) return SPEC_ERR_INVALID_ARG;
  if (B == 0 || T == 0 || n_max == 0) return SPEC_OK;
  if (!qkv || !q_out || !k_cache || !v_cache || !block_table || !prefix_len || !tree_off || !status || (rot_dim > 0 && !inv_freq))
    return SPEC_ERR_INVALID_ARG;
  if (((reinterpret_cast<uintptr_t>(qkv) | reinterpret_cast<uintptr_t>(q_out) | reinterpret_cast<uintptr_t>(k_cache) |
        reinterpret_cast<uintptr_t>(v_cache) | reinterpret_cast<uintptr_t>(q_norm) | reinterpret_cast<uintptr_t>(k_norm)) & 15) != 0)
    return SPEC_ERR_INVALID_ARG;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return SPEC_ERR_CUDA;
  RopeArgs a = {};
  a.qkv = static_cast<const char*>(qkv);
  a.row_bytes = row_stride * size;
  a.q_norm = q_norm;
  a.k_norm = k_norm;
  a.inv_freq = inv_freq;
  a.axis = axis;
  a.pos_base = pos_base;
  a.pos = pos;
  a.q_out = static_cast<char*>(q_out);
  a.k_cache = static_cast<char*>(k_cache);
  a.v_cache = static_cast<char*>(v_cache);
  a.block_table = block_table;
  a.prefix_len = prefix_len;
  a.tree_off = tree_off;
  a.status = status;
  a.eps = eps;
  a.rot = rot_dim;
  a.axes = axes;
  a.mode = pairing == SPEC_ROPE_NEIGHBOURS ? kRopeNeighbours : rot_dim / 2 % (16 / size) == 0 ? kRopeHalves : kRopeShared;
  a.max_blocks = max_blocks;
  while ((1 << a.bs_log2) < block_size) ++a.bs_log2;
  a.num_blocks = num_blocks;
  a.B = B;
  a.T = T;
  a.n_max = n_max;
  a.Hq = Hq;
  a.Hkv = Hkv;
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e;
  if (dtype == SPEC_F32) e = D == 64 ? launch_rope<float, 64>(a, sms, st) : launch_rope<float, 128>(a, sms, st);
  else e = D == 64 ? launch_rope<__nv_bfloat16, 64>(a, sms, st) : launch_rope<__nv_bfloat16, 128>(a, sms, st);
  return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}
