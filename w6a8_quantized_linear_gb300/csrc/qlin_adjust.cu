// qlin_adjust_logits: penalties for repeated tokens, biases and a grammar's mask
// on the rows of logits that sampling then reads.
#include <cmath>
#include <type_traits>

#include "qlin_ptx.cuh"
#include "qlin_step.h"

namespace qlin {
namespace {

constexpr int ADJUST_THREADS = 256;
constexpr int AHEAD = 4;              // vectors of 16 bytes in flight per thread
constexpr int MAX_SLICE = 8192;       // tokens of a block at most
constexpr int MAX_PAIRS = QLIN_MAX_TREE * QLIN_MAX_TREE / ADJUST_THREADS;

// What a block knows of a token of its slice, in a word: how often it stands in
// the history behind the prompt, its place + 1 among the slice's biases, and
// whether it stands in the prompt.
constexpr uint32_t COUNT = (1u << 20) - 1, IN_PROMPT = 1u << 31;
__device__ __forceinline__ uint32_t slot_of(uint32_t word) { return word >> 20 & 0x7FF; }

struct AdjustParams {
  qlin_adjustments a;
  const void* logits;
  void* out;
  int64_t ld, out_ld, V;
  int T, slice, cluster;
  bool in_place;
};

__device__ __forceinline__ void cluster_add(uint32_t addr, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void cluster_or(uint32_t addr, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.or.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// A sequence's penalties.
struct Penalties {
  float r, p, f;
  __device__ __forceinline__ float operator()(float x, uint32_t word, uint32_t more, const float* bias) const {
    const uint32_t n = (word & COUNT) + more;
    if (n || word & IN_PROMPT) x = x > 0.f ? __fdiv_rn(x, r) : __fmul_rn(x, r);
    if (n) x = __fsub_rn(__fsub_rn(x, __fmul_rn(f, (float)n)), p);
    const uint32_t slot = slot_of(word);
    return slot ? x + bias[slot - 1] : x;
  }
};

template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) { return __float2bfloat16(x); }

// One block per sequence and slice of the vocabulary: the slice's words first,
// from the whole history, then the slice of each of the sequence's rows in 16-byte
// vectors on the row's own alignment.  A long history is read once per cluster,
// whose blocks count for one another.
template <typename T>
__global__ void __launch_bounds__(ADJUST_THREADS) qlin_adjust_kernel(const __grid_constant__ AdjustParams p) {
  constexpr int VEC = 16 / sizeof(T);
  extern __shared__ __align__(16) uint32_t words[];  // [slice]
  __shared__ float bias[QLIN_MAX_BIAS];
  __shared__ int draft[QLIN_MAX_TREE];
  __shared__ uint32_t tree[QLIN_MAX_TREE];
  const qlin_adjustments& a = p.a;
  const int b = blockIdx.y, tid = threadIdx.x;
  const int64_t v0 = (int64_t)blockIdx.x * p.slice;
  const int n = (int)max((int64_t)0, min((int64_t)p.slice, p.V - v0));  // tokens of this slice
  pdl_wait();
  pdl_launch_dependents();
  const bool counts = a.history != nullptr, drafts = a.draft != nullptr;
  bool any_draft = false;

  // ---- the words
  if (counts || drafts || a.n_bias) {
    for (int i = tid; i < p.slice / 4; i += ADJUST_THREADS) reinterpret_cast<uint4*>(words)[i] = make_uint4(0, 0, 0, 0);
    if (drafts && tid < p.T) {
      draft[tid] = a.draft[(int64_t)b * p.T + tid];
      tree[tid] = a.mask ? (uint32_t)a.mask[b * a.tree_stride + tid] : 0xFFFFFFFFu >> (31 - tid);
    }
    if (p.cluster > 1) {
      cluster_arrive();
      cluster_wait();
    } else {
      __syncthreads();
    }
    if (counts) {
      const int32_t* h = a.history + b * a.history_stride;
      int L = a.history_len ? a.history_len[b] : a.L;
      L = max(0, min(L, a.L));
      const int prompt = a.prompt_len ? a.prompt_len[b] : 0;
      if (p.cluster == 1) {
#pragma unroll 8
        for (int i = tid; i < L; i += ADJUST_THREADS) {
          const int64_t at = h[i] - v0;
          if (at >= 0 && at < n) {
            if (i < prompt)
              atomicOr(&words[at], IN_PROMPT);
            else
              atomicAdd(&words[at], 1u);
          }
        }
      } else {
        const int rank = (int)cluster_ctarank();
        const int64_t base = v0 - (int64_t)rank * p.slice, end = min(p.V, base + (int64_t)p.slice * p.cluster);
        const uint32_t mine = smem_u32(words);
#pragma unroll 8
        for (int i = rank * ADJUST_THREADS + tid; i < L; i += p.cluster * ADJUST_THREADS) {
          const int token = h[i];
          if (token >= base && token < end) {
            const uint32_t at = (uint32_t)(token - base), owner = at / (uint32_t)p.slice;
            const uint32_t addr = dsmem_addr_u32(mine + (at - owner * p.slice) * 4, owner);
            if (i < prompt)
              cluster_or(addr, IN_PROMPT);
            else
              cluster_add(addr, 1u);
          }
        }
      }
    }
    if (p.cluster > 1) {
      cluster_arrive();
      cluster_wait();
    } else {
      __syncthreads();
    }
    if (a.n_bias && tid < 32) {  // one warp, in the list's order: biases of one token are added in that order
      const int32_t* tokens = a.bias_token + b * a.bias_stride;
      const float* values = a.bias + b * a.bias_stride;
      int used = 0;
      for (int i0 = 0; i0 < a.n_bias; i0 += 32) {
        const int i = i0 + tid;
        const int64_t at = i < a.n_bias ? tokens[i] - v0 : -1;
        const bool here = at >= 0 && at < n;
        const float value = here ? values[i] : 0.f;
        const uint32_t all = __ballot_sync(0xFFFFFFFFu, here);
        if (!all) continue;
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, here ? (int)at : -1 - tid);
        const bool first = here && (same & ((1u << tid) - 1)) == 0;
        uint32_t slot = first ? slot_of(words[at]) : 0;
        const bool fresh = first && !slot;
        const uint32_t made = __ballot_sync(0xFFFFFFFFu, fresh);
        if (fresh) {
          slot = used + __popc(made & ((1u << tid) - 1)) + 1;
          words[at] |= slot << 20;
          bias[slot - 1] = value;
        }
        used += __popc(made);
        __syncwarp();
        uint32_t again = __ballot_sync(0xFFFFFFFFu, here && !fresh);
        while (again) {
          if (tid == __ffs(again) - 1) bias[slot_of(words[at]) - 1] += value;
          again &= again - 1;
          __syncwarp();
        }
      }
    }
    any_draft = __syncthreads_or(drafts && tid < p.T && draft[tid] >= v0 && draft[tid] < v0 + n);
  }
  Penalties value = {1.f, 0.f, 0.f};
  if (a.repetition) value.r = a.repetition[b];
  if (!(value.r > 0.f)) value.r = 1.f;
  if (a.presence) value.p = a.presence[b];
  if (a.frequency) value.f = a.frequency[b];
  const bool touched_at_all = counts || a.n_bias;

  const int64_t row0 = (int64_t)b * p.T;
  auto allowed_bits = [&](int64_t row, int64_t lo, int64_t hi) -> uint32_t {  // of at most 8 tokens, the first in bit 0
    if (!a.allowed) return 0xFFFFFFFFu;
    const int32_t* w = a.allowed + row * a.allowed_stride + (lo >> 5);
    const int sh = (int)(lo & 31);
    uint32_t bits = (uint32_t)w[0] >> sh;
    if (((hi - 1) ^ lo) >> 5) bits |= (uint32_t)w[1] << (32 - sh);
    return bits;
  };

  // Tokens of the tree's rows: a row's path counts its own, on top of the history.
  // Their values are formed before anything is written, as out may be the logits.
  float path_value[MAX_PAIRS];
  bool path_here[MAX_PAIRS];
  if (any_draft) {
#pragma unroll
    for (int k = 0; k < MAX_PAIRS; k++) {
      const int pair = tid + k * ADJUST_THREADS, t = pair / p.T, j = pair % p.T;
      path_here[k] = false;
      if (t >= p.T || !(tree[t] >> j & 1) || draft[j] < v0 || draft[j] >= v0 + n) continue;
      uint32_t more = 0;
      bool first = true;
      for (int i = 0; i < p.T; i++)
        if (tree[t] >> i & 1 && draft[i] == draft[j]) {
          more++;
          if (i < j) first = false;
        }
      if (!first || !(allowed_bits(row0 + t, draft[j], (int64_t)draft[j] + 1) & 1)) continue;
      const T* in = static_cast<const T*>(p.logits) + (row0 + t) * p.ld;
      path_value[k] = value(to_float(in[draft[j]]), words[draft[j] - v0], more, bias);
      path_here[k] = true;
    }
    if (p.in_place) __syncthreads();
  }

  // ---- the rows
  const T forbidden = from_float<T>(-INFINITY);
  const int vectors = p.slice / VEC + 1;  // of a row, on its alignment
  if (!p.in_place || touched_at_all || a.allowed) {
    const int total = n ? vectors * p.T : 0;
    for (int i0 = tid; i0 < total; i0 += AHEAD * ADJUST_THREADS) {
      uint4 x[AHEAD];
      uint32_t bits[AHEAD];
      int lo[AHEAD], hi[AHEAD];  // places of a vector's tokens in the slice; lo = hi: none
      bool whole[AHEAD];
      const T* src[AHEAD];
      T* dst[AHEAD];
#pragma unroll
      for (int u = 0; u < AHEAD; u++) {
        const int i = i0 + u * ADJUST_THREADS;
        lo[u] = hi[u] = 0;
        if (i >= total) continue;
        const int t = i / vectors, v = i - t * vectors;
        src[u] = static_cast<const T*>(p.logits) + (row0 + t) * p.ld + v0;
        dst[u] = static_cast<T*>(p.out) + (row0 + t) * p.out_ld + v0;
        const int shift = (int)(reinterpret_cast<uintptr_t>(src[u]) / sizeof(T) % VEC);
        const int e = v * VEC - shift;
        lo[u] = max(e, 0), hi[u] = min(e + VEC, n);
        if (lo[u] >= hi[u]) {
          lo[u] = hi[u] = 0;
          continue;
        }
        whole[u] = hi[u] - lo[u] == VEC && reinterpret_cast<uintptr_t>(dst[u] + lo[u]) % 16 == 0;
        bits[u] = allowed_bits(row0 + t, v0 + lo[u], v0 + hi[u]) | ~((1u << (hi[u] - lo[u])) - 1);
        const bool none = !(bits[u] & ((1u << (hi[u] - lo[u])) - 1));
        if (whole[u] && !none && !p.in_place) x[u] = *reinterpret_cast<const uint4*>(src[u] + lo[u]);
      }
#pragma unroll
      for (int u = 0; u < AHEAD; u++) {
        if (lo[u] >= hi[u]) continue;
        uint32_t any = 0;
        if (touched_at_all)
          for (int e = lo[u]; e < hi[u]; e++) any |= words[e];
        if (p.in_place && !any && bits[u] == 0xFFFFFFFFu) continue;
        if (whole[u]) {
          if (p.in_place) x[u] = *reinterpret_cast<const uint4*>(src[u] + lo[u]);
          if (any || bits[u] != 0xFFFFFFFFu) {
            T y[VEC];
            *reinterpret_cast<uint4*>(y) = x[u];
#pragma unroll
            for (int e = 0; e < VEC; e++) {
              const uint32_t word = any ? words[lo[u] + e] : 0;
              if (word) y[e] = from_float<T>(value(to_float(y[e]), word, 0, bias));
              if (!(bits[u] >> e & 1)) y[e] = forbidden;
            }
            x[u] = *reinterpret_cast<const uint4*>(y);
          }
          *reinterpret_cast<uint4*>(dst[u] + lo[u]) = x[u];
        } else {
          for (int e = lo[u]; e < hi[u]; e++) {
            T y = src[u][e];
            const uint32_t word = any ? words[e] : 0;
            if (word) y = from_float<T>(value(to_float(y), word, 0, bias));
            if (!(bits[u] >> (e - lo[u]) & 1)) y = forbidden;
            dst[u][e] = y;
          }
        }
      }
    }
  }
  if (any_draft) {
    __syncthreads();
#pragma unroll
    for (int k = 0; k < MAX_PAIRS; k++) {
      const int pair = tid + k * ADJUST_THREADS, t = pair / p.T, j = pair % p.T;
      if (path_here[k]) static_cast<T*>(p.out)[(row0 + t) * p.out_ld + draft[j]] = from_float<T>(path_value[k]);
    }
  }
}

}  // namespace
}  // namespace qlin

using namespace qlin;

extern "C" qlin_status qlin_adjust_logits(int B, int T, int64_t V, int dtype, const void* logits, int64_t ld, void* out,
                                          int64_t out_ld, const qlin_adjustments* adjustments, unsigned flags,
                                          void* stream) {
  if (B < 0 || T < 0 || V < 1 || (dtype != QLIN_F32 && dtype != QLIN_BF16) || !adjustments) return QLIN_ERR_INVALID_ARG;
  qlin_adjustments a = *adjustments;
  if (flags & ~QLIN_FLAG_PDL) return QLIN_ERR_INVALID_ARG;
  if (a.L < 0 || a.n_bias < 0) return QLIN_ERR_INVALID_ARG;
  if (V > QLIN_SAMPLE_MAX_V || B > 65535 || (int64_t)B * T > (1 << 24) || a.L > QLIN_MAX_HISTORY ||
      a.n_bias > QLIN_MAX_BIAS || (a.draft && T > QLIN_MAX_TREE))
    return QLIN_ERR_UNSUPPORTED;
  if (B == 0 || T == 0) return QLIN_OK;
  const int64_t size = dtype == QLIN_F32 ? 4 : 2, M = (int64_t)B * T;
  if (!logits || !out || !is_aligned(logits, size) || !is_aligned(out, size) || ld < V || out_ld < V)
    return QLIN_ERR_INVALID_ARG;
  for (const void* x : {(const void*)a.history, (const void*)a.history_len, (const void*)a.prompt_len, (const void*)a.draft,
                        (const void*)a.mask, (const void*)a.repetition, (const void*)a.presence, (const void*)a.frequency,
                        (const void*)a.bias_token, (const void*)a.bias, (const void*)a.allowed})
    if (!is_aligned(x, 4)) return QLIN_ERR_INVALID_ARG;
  if (a.L && (!a.history || a.history_stride < a.L)) return QLIN_ERR_INVALID_ARG;
  if (a.n_bias && (!a.bias_token || !a.bias || (a.bias_stride != 0 && a.bias_stride < a.n_bias)))
    return QLIN_ERR_INVALID_ARG;
  if (a.draft && (a.tree_stride < 0 || (a.tree_stride != 0 && a.tree_stride < T))) return QLIN_ERR_INVALID_ARG;
  if (a.allowed && a.allowed_stride != 0 && a.allowed_stride < (V + 31) / 32) return QLIN_ERR_INVALID_ARG;
  AdjustParams p = {};
  p.in_place = out == logits && out_ld == ld;
  if (!p.in_place && rows_overlap(out, out_ld * size, V * size, logits, ld * size, V * size, M)) return QLIN_ERR_INVALID_ARG;
  if (!a.repetition && !a.presence && !a.frequency) a.history = nullptr, a.draft = nullptr;  // nothing comes of them
  if (!a.L) a.history = nullptr;
  p.a = a;
  p.logits = logits, p.out = out, p.ld = ld, p.out_ld = out_ld, p.V = V, p.T = T;
  int64_t slice = (V * B + 911) / 912;
  slice = slice < 512 ? 512 : slice > MAX_SLICE ? MAX_SLICE : (slice + 127) / 128 * 128;
  int64_t slices = (V + slice - 1) / slice;
  p.slice = (int)slice;
  p.cluster = a.history && a.L > 4096 && slices > 1 ? 8 : 1;
  slices = (slices + p.cluster - 1) / p.cluster * p.cluster;
  void* args[] = {&p};
  const void* fn = dtype == QLIN_F32 ? reinterpret_cast<const void*>(qlin_adjust_kernel<float>)
                                     : reinterpret_cast<const void*>(qlin_adjust_kernel<__nv_bfloat16>);
  return launch_step(fn, dim3((unsigned)slices, (unsigned)B, 1), dim3(ADJUST_THREADS, 1, 1), (size_t)slice * 4,
                     static_cast<cudaStream_t>(stream), args, (flags & QLIN_FLAG_PDL) != 0, p.cluster);
}
