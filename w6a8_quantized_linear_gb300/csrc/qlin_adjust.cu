// qlin_adjust_logits: penalties for repeated tokens, biases and a grammar's mask
// on the rows of logits that sampling then reads.
#include <cmath>
#include <mutex>

#include "qlin_ptx.cuh"
#include "qlin_step.h"

namespace qlin {
namespace {

constexpr int ADJUST_THREADS = 256;
constexpr int AHEAD = 4;              // vectors of 16 bytes in flight per thread
constexpr int HISTORY_AHEAD = 8;      // tokens of the history in flight per thread
constexpr int MAX_SLICE = 16384;      // tokens of a block at most
constexpr int CLUSTER = 8;            // blocks that share the reading of a long history
constexpr int LONG_HISTORY = 4096;
constexpr int CLUSTER_SLICE = 2048;   // tokens of a block of theirs at most: each counts for all eight
constexpr int ROWS = QLIN_MAX_TREE;   // rows of a block at most
constexpr int MAX_PAIRS = ROWS * ROWS / ADJUST_THREADS;

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
  int column;        // words between the eight columns that a slice's words lie in
  uint32_t inverse;  // 2^32 / (vectors of a row), rounded up
  bool in_place;
};

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

// One block per sequence, slice of the vocabulary and (at most 32 of its) rows: the
// slice's words first, from the whole history, then the rows' slices in 16-byte
// vectors on their own alignment, whose first loads are on their way meanwhile.  A
// long history is read once per cluster: each block counts a part of it for all
// slices of the cluster, and adds up its own slice's counts from all blocks.
// Word i of a slice lies in column i % 8 (so that vectors' words fall into
// different banks), and a bit per token says which words are not zero.
template <typename T>
__global__ void __launch_bounds__(ADJUST_THREADS) qlin_adjust_kernel(const __grid_constant__ AdjustParams p) {
  constexpr int VEC = 16 / sizeof(T);
  extern __shared__ __align__(16) uint32_t shared[];  // words of the cluster's slices, bits of this one
  __shared__ float bias[QLIN_MAX_BIAS];
  __shared__ int draft[ROWS];
  __shared__ uint32_t tree[ROWS];
  const qlin_adjustments& a = p.a;
  const int b = blockIdx.y, tid = threadIdx.x, S = p.slice, column = p.column;
  const int rank = p.cluster > 1 ? (int)cluster_ctarank() : 0;
  const int t0 = blockIdx.z * ROWS, rows = min(p.T - t0, ROWS);
  const int64_t v0 = (int64_t)blockIdx.x * S;
  const int n = (int)max((int64_t)0, min((int64_t)S, p.V - v0));  // tokens of this slice
  uint32_t* words = shared + rank * 8 * column;
  uint32_t* bits = shared + p.cluster * 8 * column;
  auto place = [column](int i) { return (i & 7) * column + (i >> 3); };
  pdl_wait();
  pdl_launch_dependents();
  const bool counts = a.history != nullptr, drafts = a.draft != nullptr;
  const int64_t row0 = (int64_t)b * p.T + t0;

  auto allowed_bits = [&](int64_t row, int64_t lo, int64_t hi) -> uint32_t {  // of at most 8 tokens, the first in bit 0
    const int32_t* w = a.allowed + row * a.allowed_stride + (lo >> 5);
    const int sh = (int)(lo & 31);
    uint32_t m = (uint32_t)w[0] >> sh;
    if (((hi - 1) ^ lo) >> 5) m |= (uint32_t)w[1] << (32 - sh);
    return m;
  };

  // ---- vectors of the rows: which, and what is loaded of them ahead
  const int vectors = S / VEC + 1, total = n ? vectors * rows : 0;
  struct Vector {
    const T* src;
    T* dst;
    int t, lo, hi;  // its tokens' places in the slice
    bool whole;     // 16 bytes on both sides
  };
  auto vector = [&](int i) {
    Vector v;
    v.t = rows > 1 ? (int)__umulhi((uint32_t)i, p.inverse) : 0;
    v.src = static_cast<const T*>(p.logits) + (row0 + v.t) * p.ld + v0;
    v.dst = static_cast<T*>(p.out) + (row0 + v.t) * p.out_ld + v0;
    const int e = (i - v.t * vectors) * VEC - (int)(reinterpret_cast<uintptr_t>(v.src) / sizeof(T) % VEC);
    v.lo = max(e, 0), v.hi = i < total ? min(e + VEC, n) : 0;
    v.whole = v.hi - v.lo == VEC && reinterpret_cast<uintptr_t>(v.dst + v.lo) % 16 == 0;
    return v;
  };
  uint4 x[AHEAD];
  uint32_t open[AHEAD];  // allowed tokens
  auto load = [&](int i0) {
#pragma unroll
    for (int u = 0; u < AHEAD; u++) {
      const Vector v = vector(i0 + u * ADJUST_THREADS);
      open[u] = 0xFFFFFFFFu;
      if (v.lo >= v.hi) continue;
      const uint32_t behind = 0xFFFFFFFFu << (v.hi - v.lo);
      if (a.allowed) open[u] = allowed_bits(row0 + v.t, v0 + v.lo, v0 + v.hi) | behind;
      if (v.whole && !p.in_place && open[u] != behind) x[u] = *reinterpret_cast<const uint4*>(v.src + v.lo);
    }
  };
  load(tid);

  // ---- the words
  bool any_draft = false;
  if (counts || drafts || a.n_bias) {
    const int32_t* h = counts ? a.history + b * a.history_stride : nullptr;
    const int step = p.cluster * ADJUST_THREADS, h0 = rank * ADJUST_THREADS + tid;
    int token[HISTORY_AHEAD];
    auto read = [&](int i0) {
#pragma unroll
      for (int u = 0; u < HISTORY_AHEAD; u++) token[u] = i0 + u * step < a.L ? h[i0 + u * step] : -1;
    };
    if (counts) read(h0);
    int L = a.L, prompt = 0;
    if (counts) {
      if (a.history_len) L = max(0, min(a.history_len[b], L));
      if (a.prompt_len) prompt = a.prompt_len[b];
    }
    const int32_t* bias_token = a.bias_token + b * a.bias_stride;
    int first_bias = tid < 32 && tid < a.n_bias ? bias_token[tid] : -1;
    if (drafts && tid < p.T) {
      draft[tid] = a.draft[(int64_t)b * p.T + tid];
      tree[tid] = a.mask ? (uint32_t)a.mask[b * a.tree_stride + tid] : 0xFFFFFFFFu >> (31 - tid);
    }
    for (int i = tid; i < (p.cluster * 8 * column + S / 32 + 3) / 4; i += ADJUST_THREADS)
      reinterpret_cast<uint4*>(shared)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    if (counts) {
      const int64_t base = v0 - (int64_t)rank * S;
      const int range = p.cluster > 1 ? S * p.cluster : n;
#pragma unroll 1
      for (int i0 = h0; i0 < L; i0 += HISTORY_AHEAD * step) {
        if (i0 != h0) read(i0);
#pragma unroll
        for (int u = 0; u < HISTORY_AHEAD; u++) {
          const int i = i0 + u * step;
          const int64_t at = token[u] - base;
          if (i >= L || at < 0 || at >= range || token[u] >= p.V) continue;
          uint32_t* word;
          if (p.cluster > 1) {
            const uint32_t owner = (uint32_t)at / (uint32_t)S;
            word = shared + owner * 8 * column + place((int)at - owner * S);
          } else {
            word = words + place((int)at);
            atomicOr(&bits[at >> 5], 1u << (at & 31));
          }
          if (i < prompt)
            atomicOr(word, IN_PROMPT);
          else
            atomicAdd(word, 1u);
        }
      }
      if (p.cluster > 1) {
        cluster_arrive();
        cluster_wait();
        // all lanes of a warp stay: a ballot per 32 tokens
        for (int i = tid; i < S; i += ADJUST_THREADS) {
          const uint32_t mine = smem_u32(words + place(i));
          uint32_t sum = 0;
#pragma unroll
          for (int r = 0; r < CLUSTER; r++) {
            uint32_t w;
            asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(w) : "r"(dsmem_addr_u32(mine, r)) : "memory");
            sum = ((sum & ~IN_PROMPT) + (w & ~IN_PROMPT)) | ((sum | w) & IN_PROMPT);
          }
          words[place(i)] = sum;  // read by this block alone
          const uint32_t any = __ballot_sync(0xFFFFFFFFu, sum != 0);
          if ((tid & 31) == 0) bits[i >> 5] = any;
        }
        cluster_arrive();  // waited for at the end: no block leaves while others read its words
      }
      __syncthreads();
    }
    if (a.n_bias && tid < 32) {  // one warp, in the list's order: biases of one token are added in that order
      const float* values = a.bias + b * a.bias_stride;
      int used = 0;
      for (int i0 = 0; i0 < a.n_bias; i0 += 32) {
        const int i = i0 + tid;
        const int64_t at = i < a.n_bias ? (i0 ? bias_token[i] : first_bias) - v0 : -1;
        const bool here = at >= 0 && at < n;
        const uint32_t all = __ballot_sync(0xFFFFFFFFu, here);
        if (!all) continue;
        const float value = here ? values[i] : 0.f;
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, here ? (int)at : -1 - tid);
        const bool first = here && (same & ((1u << tid) - 1)) == 0;
        uint32_t* word = words + place(here ? (int)at : 0);
        uint32_t slot = first ? slot_of(*word) : 0;
        const bool fresh = first && !slot;
        const uint32_t made = __ballot_sync(0xFFFFFFFFu, fresh);
        if (fresh) {
          slot = used + __popc(made & ((1u << tid) - 1)) + 1;
          *word |= slot << 20;
          atomicOr(&bits[at >> 5], 1u << (at & 31));
          bias[slot - 1] = value;
        }
        used += __popc(made);
        __syncwarp();
        uint32_t again = __ballot_sync(0xFFFFFFFFu, here && !fresh);
        while (again) {
          if (tid == __ffs(again) - 1) bias[slot_of(*word) - 1] += value;
          again &= again - 1;
          __syncwarp();
        }
      }
    }
    if (a.n_bias || drafts) any_draft = __syncthreads_or(drafts && tid < p.T && draft[tid] >= v0 && draft[tid] < v0 + n);
  }
  Penalties value = {1.f, 0.f, 0.f};
  if (a.repetition) value.r = a.repetition[b];
  if (!(value.r > 0.f)) value.r = 1.f;
  if (a.presence) value.p = a.presence[b];
  if (a.frequency) value.f = a.frequency[b];
  const bool touched_at_all = counts || a.n_bias;

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
      if (!first || (a.allowed && !(allowed_bits(row0 + t, draft[j], (int64_t)draft[j] + 1) & 1))) continue;
      const T* in = static_cast<const T*>(p.logits) + (row0 + t) * p.ld;
      path_value[k] = value(to_float(in[draft[j]]), words[place((int)(draft[j] - v0))], more, bias);
      path_here[k] = true;
    }
    if (p.in_place) __syncthreads();
  }

  // ---- the rows
  const T forbidden = from_float<T>(-INFINITY);
  if (!p.in_place || touched_at_all || a.allowed) {
#pragma unroll 1
    for (int i0 = tid; i0 < total; i0 += AHEAD * ADJUST_THREADS) {
      if (i0 != tid) load(i0);
#pragma unroll
      for (int u = 0; u < AHEAD; u++) {
        const Vector v = vector(i0 + u * ADJUST_THREADS);
        if (v.lo >= v.hi) continue;
        uint32_t any = 0;
        if (touched_at_all) {
          any = bits[v.lo >> 5] >> (v.lo & 31);
          if ((v.hi - 1) >> 5 != v.lo >> 5) any |= bits[(v.hi - 1) >> 5] << (32 - (v.lo & 31));
          any &= ~(0xFFFFFFFFu << (v.hi - v.lo));
        }
        if (p.in_place && !any && open[u] == 0xFFFFFFFFu) continue;
        if (v.whole) {
          if (p.in_place) x[u] = *reinterpret_cast<const uint4*>(v.src + v.lo);
          if (any || open[u] != 0xFFFFFFFFu) {
            T y[VEC];
            *reinterpret_cast<uint4*>(y) = x[u];
#pragma unroll
            for (int e = 0; e < VEC; e++) {
              if (any >> e & 1) y[e] = from_float<T>(value(to_float(y[e]), words[place(v.lo + e)], 0, bias));
              if (!(open[u] >> e & 1)) y[e] = forbidden;
            }
            x[u] = *reinterpret_cast<const uint4*>(y);
          }
          *reinterpret_cast<uint4*>(v.dst + v.lo) = x[u];
        } else {
          for (int e = 0; e < v.hi - v.lo; e++) {
            T y = v.src[v.lo + e];
            if (any >> e & 1) y = from_float<T>(value(to_float(y), words[place(v.lo + e)], 0, bias));
            if (!(open[u] >> e & 1)) y = forbidden;
            v.dst[v.lo + e] = y;
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
  if (p.cluster > 1) cluster_wait();
}

struct AdjustDevice {
  std::once_flag once;
  qlin_status ready = QLIN_ERR_CUDA;
  int sms = 0;
};
AdjustDevice g_adjust[64];

constexpr int64_t column_of(int64_t slice) { return (slice / 8 + 27) / 32 * 32 + 4; }  // banks: 4 more per column
constexpr int64_t adjust_smem(int64_t slice, int cluster) { return (cluster * 8 * column_of(slice) + slice / 32 + 4) * 4; }

const void* adjust_fn(int dtype) {
  return dtype == QLIN_F32 ? reinterpret_cast<const void*>(qlin_adjust_kernel<float>)
                           : reinterpret_cast<const void*>(qlin_adjust_kernel<__nv_bfloat16>);
}

qlin_status adjust_setup(int* sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return status_of(e);
  if (dev < 0 || dev >= 64) return QLIN_ERR_CUDA;
  AdjustDevice& d = g_adjust[dev];
  std::call_once(d.once, [&d, dev] {
    cudaError_t e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
    const int64_t one = adjust_smem(MAX_SLICE, 1), many = adjust_smem(CLUSTER_SLICE, CLUSTER);
    for (int dtype : {QLIN_F32, QLIN_BF16})
      if (e == cudaSuccess)
        e = cudaFuncSetAttribute(adjust_fn(dtype), cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(one > many ? one : many));
    d.ready = d.sms > 0 ? status_of(e) : QLIN_ERR_CUDA;
  });
  *sms = d.sms;
  return d.ready;
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
  if (V > QLIN_SAMPLE_MAX_V || B > 65535 || T > 65535 * ROWS || (int64_t)B * T > (1 << 24) || a.L > QLIN_MAX_HISTORY ||
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
  int sms = 0;
  const qlin_status st = adjust_setup(&sms);
  if (st != QLIN_OK) return st;
  p.cluster = a.history && a.L > LONG_HISTORY && V > 4096 ? CLUSTER : 1;
  const int64_t most = p.cluster > 1 ? CLUSTER_SLICE : MAX_SLICE;
  int64_t slice = (V * B + 3 * sms - 1) / (3 * sms);
  slice = slice < 512 ? 512 : slice > most ? most : (slice + 127) / 128 * 128;
  int64_t slices = (V + slice - 1) / slice;
  slices = (slices + p.cluster - 1) / p.cluster * p.cluster;
  p.slice = (int)slice;
  p.column = (int)column_of(slice);
  const int64_t vectors = slice * size / 16 + 1;
  p.inverse = (uint32_t)(((1ull << 32) + vectors - 1) / vectors);
  void* args[] = {&p};
  return launch_step(adjust_fn(dtype), dim3((unsigned)slices, (unsigned)B, (unsigned)((T + ROWS - 1) / ROWS)),
                     dim3(ADJUST_THREADS, 1, 1), (size_t)adjust_smem(slice, p.cluster), static_cast<cudaStream_t>(stream),
                     args, (flags & QLIN_FLAG_PDL) != 0, p.cluster);
}
