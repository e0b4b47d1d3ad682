// qlin_adjust_logits: penalties for repeated tokens, biases and a grammar's mask
// on the rows of logits that sampling then reads.
#include <algorithm>
#include <cmath>
#include <mutex>

#include "qlin_ptx.cuh"
#include "qlin_step.h"

namespace qlin {
namespace {

constexpr int ADJUST_THREADS = 512;
constexpr int BLOCKS = 2;             // per SM
constexpr int AHEAD = 4;              // vectors of 16 bytes in flight per thread
constexpr int HISTORY_AHEAD = 8;      // tokens of the history in flight per thread
constexpr int FIXES_AHEAD = 4;        // changed logits in flight per thread
constexpr int CLUSTER = 4;            // blocks that share the reading of a long history
constexpr int LONG_HISTORY = 4096, VERY_LONG_HISTORY = 32768;
constexpr int64_t CLUSTER_SLICE = 4096;  // tokens of a block of theirs at most: each counts for all of them
constexpr int ROWS = QLIN_MAX_TREE;   // rows of a block at most
constexpr int MAX_PAIRS = ROWS * ROWS / ADJUST_THREADS;

// What a block knows of a token of its slice, in a word: how often it stands in
// the history behind the prompt, the place + 1 of its first bias among the
// slice's, and whether it stands in the prompt.
constexpr uint32_t COUNT = (1u << 20) - 1, IN_PROMPT = 1u << 31;
__device__ __forceinline__ uint32_t slot_of(uint32_t word) { return word >> 20 & 0x7FF; }

struct AdjustParams {
  qlin_adjustments a;
  const void* logits;
  void* out;
  int64_t ld, out_ld, V;
  int T, slice;
  int vectors;              // of a row's slice, on the row's alignment
  uint32_t vectors_inverse; // 2^32 / vectors, rounded up
  bool in_place, history_vectors;
  bool aligned;             // every row of both on the 16-byte grid
};

// One row per sequence, several, or a tree's drafted ones.
enum class Rows { ONE, SEVERAL, DRAFTED };

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

// One block per sequence, slice of the vocabulary and (at most 32 of its) rows.  The
// slice's words are formed first, from the whole history, and with them a list of
// the tokens that they concern, few of the slice's as a rule.  The rows' slices
// are copied meanwhile, in 16-byte vectors on their own alignment and without what
// is forbidden, and in the end the listed tokens' logits are written, a thread
// each: looked for within the vectors they cost a warp its time wherever one lane
// has one (64 rows of 262144 in bf16: 47 us).  A long history is read once per
// cluster: each block counts a part of it for all slices of the cluster, and adds
// up its own slice's counts.  A block that nothing concerns leaves behind the copy.
//
// Without a history the copy runs at the memory's rate: 64 rows of 262144 in bf16,
// 67 MB, 11.8 us.  With 4096 tokens of history 23.9 us: per block the tokens, the
// counts, the listed logits and their way back are waited for one after the other,
// by two blocks per SM (registers), four rounds of them.  Blocks that stay and go
// through slices with the next one's vectors on their way took 33 us (spills, and
// fewer phases side by side); three blocks per SM, 28.
// 8 rows of 131071 with a history of 20011 tokens 13 us (the cluster's barrier and
// sums 5 of them; 15.6 with every block reading it all), one row of 32000 3.7 us.
// Biases found by the whole block and blocks that leave early cost the 64 rows 0.9
// of their us, for 4.9 of 12.9 with 300 biases and 1.5 of 21.7 with 30 rows of 200321.
template <typename T, bool CLUSTERS, Rows KIND>
__global__ void __launch_bounds__(ADJUST_THREADS, BLOCKS) qlin_adjust_kernel(const __grid_constant__ AdjustParams p) {
  constexpr int VEC = 16 / sizeof(T), C = CLUSTERS ? CLUSTER : 1;
  constexpr bool DRAFTS = KIND == Rows::DRAFTED, ONE = KIND == Rows::ONE;
  extern __shared__ __align__(16) uint32_t shared[];  // words of the cluster's slices, the list of this one
  __shared__ float bias[QLIN_MAX_BIAS];
  __shared__ uint16_t bias_at[QLIN_MAX_BIAS];
  __shared__ int bias_hits[ADJUST_THREADS / 32];
  __shared__ int draft[ROWS];
  __shared__ uint32_t tree[ROWS];
  __shared__ int listed;
  __shared__ uint16_t queues[ADJUST_THREADS / 32][32 * HISTORY_AHEAD];
  const qlin_adjustments& a = p.a;
  const int b = blockIdx.y, tid = threadIdx.x, S = p.slice, V = (int)p.V;
  const int rank = CLUSTERS ? (int)cluster_ctarank() : 0;
  const int t0 = ONE ? 0 : blockIdx.z * ROWS, rows = ONE ? 1 : min(p.T - t0, ROWS);
  const int v0 = blockIdx.x * S, n = max(0, min(S, V - v0));  // tokens of this slice
  uint32_t* words = shared + rank * S;
  uint16_t* list = reinterpret_cast<uint16_t*>(shared + C * S);
  pdl_wait();
  pdl_launch_dependents();
  const bool counts = a.history != nullptr;
  const int64_t row0 = (int64_t)b * p.T + t0;

  auto allowed_bits = [&](int t, int lo, int hi) -> uint32_t {  // of at most 8 tokens of the slice, the first in bit 0
    lo += v0, hi += v0;
    const int32_t* w = a.allowed + (row0 + t) * a.allowed_stride + (lo >> 5);
    uint32_t m = (uint32_t)w[0] >> (lo & 31);
    if (((hi - 1) ^ lo) >> 5) m |= (uint32_t)w[1] << (32 - (lo & 31));
    return m;
  };

  // ---- vectors of the rows
  const int total = n ? p.vectors * rows : 0;
  struct Vector {
    const T* src;
    T* dst;
    int t, lo, hi;  // its row, its tokens' places in the slice
    bool whole;     // 16 bytes on both sides
  };
  auto vector = [&](int i) {
    Vector v;
    v.t = ONE ? 0 : (int)__umulhi((uint32_t)i, p.vectors_inverse);
    v.src = static_cast<const T*>(p.logits) + (row0 + v.t) * p.ld + v0;
    v.dst = static_cast<T*>(p.out) + (row0 + v.t) * p.out_ld + v0;
    const int shift = (int)(reinterpret_cast<uintptr_t>(v.src) / sizeof(T) % VEC);
    const int out_shift = (int)(reinterpret_cast<uintptr_t>(v.dst) / sizeof(T) % VEC);
    const int e = (i - v.t * p.vectors) * VEC - shift;
    v.lo = max(e, 0), v.hi = i < total ? min(e + VEC, n) : 0;
    v.whole = v.hi - v.lo == VEC && shift == out_shift;
    return v;
  };
  uint4 x[AHEAD];
  uint32_t open[AHEAD];  // allowed tokens
  const T* const src = static_cast<const T*>(p.logits) + row0 * p.ld + v0;
  T* const dst = static_cast<T*>(p.out) + row0 * p.out_ld + v0;
  const T forbidden = from_float<T>(-INFINITY);
  const bool plain = ONE && p.aligned && !a.allowed, idle = p.in_place && !a.allowed;
  auto load = [&](int i0) {
#pragma unroll
    for (int u = 0; u < AHEAD; u++) {
      const Vector v = vector(i0 + u * ADJUST_THREADS);
      open[u] = 0xFFFFFFFFu;
      if (v.lo >= v.hi) continue;
      const uint32_t behind = 0xFFFFFFFFu << (v.hi - v.lo);
      if (a.allowed) open[u] = allowed_bits(v.t, v.lo, v.hi) | behind;
      if (v.whole && !p.in_place && open[u] != behind) x[u] = *reinterpret_cast<const uint4*>(v.src + v.lo);
    }
  };
  if (plain && !idle) {
#pragma unroll
    for (int u = 0; u < AHEAD; u++)
      if (tid + u * ADJUST_THREADS < n / VEC) x[u] = reinterpret_cast<const uint4*>(src)[tid + u * ADJUST_THREADS];
  } else if (!idle) {
    load(tid);
  }

  // ---- the rows, without what is forbidden (as the words below do not concern them)
  auto copy = [&] {
    if (idle) return;
    if (plain) {  // at most AHEAD vectors a thread
#pragma unroll
      for (int u = 0; u < AHEAD; u++)
        if (tid + u * ADJUST_THREADS < n / VEC) reinterpret_cast<uint4*>(dst)[tid + u * ADJUST_THREADS] = x[u];
      if (tid < n % VEC) dst[n / VEC * VEC + tid] = src[n / VEC * VEC + tid];
      return;
    }
#pragma unroll 1
    for (int i0 = tid; i0 < total; i0 += AHEAD * ADJUST_THREADS) {
      if (i0 != tid) load(i0);
#pragma unroll
      for (int u = 0; u < AHEAD; u++) {
        const Vector v = vector(i0 + u * ADJUST_THREADS);
        if (v.lo >= v.hi || (p.in_place && open[u] == 0xFFFFFFFFu)) continue;
        if (v.whole) {
          if (p.in_place) x[u] = *reinterpret_cast<const uint4*>(v.src + v.lo);
          if (open[u] != 0xFFFFFFFFu) {
            T z[VEC];
            *reinterpret_cast<uint4*>(z) = x[u];
#pragma unroll
            for (int e = 0; e < VEC; e++)
              if (!(open[u] >> e & 1)) z[e] = forbidden;
            x[u] = *reinterpret_cast<const uint4*>(z);
          }
          *reinterpret_cast<uint4*>(v.dst + v.lo) = x[u];
        } else {
          for (int e = 0; e < v.hi - v.lo; e++) v.dst[v.lo + e] = open[u] >> e & 1 ? v.src[v.lo + e] : forbidden;
        }
      }
    }
  };

  // ---- the words and their list
  bool any_draft = false;
  int fixes = 0;
  if (counts || DRAFTS || a.n_bias) {
    int first_bias = -1;
    float first_value = 0.f;
    if (tid < a.n_bias)
      first_bias = a.bias_token[b * a.bias_stride + tid], first_value = a.bias[b * a.bias_stride + tid];
    bool concerned = CLUSTERS || a.n_bias > ADJUST_THREADS;  // something here concerns this slice, as far as this thread knows
    if (DRAFTS && tid < p.T) {
      draft[tid] = a.draft[(int64_t)b * p.T + tid];
      concerned |= draft[tid] >= 0 && (uint32_t)(draft[tid] - v0) < (uint32_t)n;
      tree[tid] = a.mask ? (uint32_t)a.mask[b * a.tree_stride + tid] : 0xFFFFFFFFu >> (31 - tid);
    }
    if (tid == 0) listed = 0;
    // Biases of the slice, in the list's order: their places and values.  (Found
    // before a barrier and held behind it; counted among the warps in between.)
    int held = 0;
    bool bias_here = false;
    uint32_t bias_lanes = 0;
    auto find_biases = [&] {
      bias_here = first_bias >= 0 && (uint32_t)(first_bias - v0) < (uint32_t)n;
      bias_lanes = __ballot_sync(0xFFFFFFFFu, bias_here);
      if ((tid & 31) == 0) bias_hits[tid >> 5] = __popc(bias_lanes);
    };
    auto hold_biases = [&] {
      if (a.n_bias <= 32) {  // the first warp's alone
        if (bias_here) {
          const int k = __popc(bias_lanes & ((1u << tid) - 1));
          bias_at[k] = (uint16_t)(first_bias - v0);
          bias[k] = first_value;
        }
        held = __popc(bias_lanes);
        return;
      }
      const int of_warp = bias_hits[tid & (ADJUST_THREADS / 32 - 1)], lane = tid & 31;
      const int before = __reduce_add_sync(0xFFFFFFFFu, lane < (tid >> 5) ? of_warp : 0);
      if (bias_here) {
        const int k = held + before + __popc(bias_lanes & ((1u << lane) - 1));
        bias_at[k] = (uint16_t)(first_bias - v0);
        bias[k] = first_value;
      }
      held += __reduce_add_sync(0xFFFFFFFFu, lane < ADJUST_THREADS / 32 ? of_warp : 0);
    };
    auto clear = [&] {
      for (int i = tid; i < C * S / 4; i += ADJUST_THREADS) reinterpret_cast<uint4*>(shared)[i] = make_uint4(0, 0, 0, 0);
      copy();
      if (a.n_bias) find_biases();
      if (!__syncthreads_or(concerned || bias_here)) return false;
      if (a.n_bias) hold_biases();
      return true;
    };
    if (counts) {
      // a thread takes four tokens in a row, HISTORY_AHEAD on their way
      const int32_t* h = a.history + b * a.history_stride;
      int token[HISTORY_AHEAD], L = a.L, prompt = 0;
      constexpr int ROUND = C * ADJUST_THREADS * HISTORY_AHEAD;
      auto ahead = [](int u) { return u / 4 * (C * ADJUST_THREADS * 4) + u % 4; };
      int h0 = (rank * ADJUST_THREADS + tid) * 4;  // this thread's first token of the round
      auto read = [&] {
        if (p.history_vectors) {
#pragma unroll
          for (int u = 0; u < HISTORY_AHEAD; u += 4) {
            const int4 q = h0 + ahead(u) < a.L ? *reinterpret_cast<const int4*>(h + h0 + ahead(u)) : make_int4(-1, -1, -1, -1);
            token[u] = q.x, token[u + 1] = q.y, token[u + 2] = q.z, token[u + 3] = q.w;
          }
        } else {
#pragma unroll
          for (int u = 0; u < HISTORY_AHEAD; u++) token[u] = h0 + ahead(u) < a.L ? h[h0 + ahead(u)] : -1;
        }
      };
      read();
      if (a.history_len) L = max(0, min(a.history_len[b], L));
      if (a.prompt_len) prompt = max(0, a.prompt_len[b]);
      const int base = v0 - rank * S;
      const uint32_t range = CLUSTERS ? (uint32_t)min(C * S, V - base) : (uint32_t)n;
      concerned |= L > ROUND;
#pragma unroll
      for (int u = 0; u < HISTORY_AHEAD; u++)
        concerned |= (uint32_t)token[u] - (uint32_t)base < range && ahead(u) < L - h0;
      if (!clear()) return;  // (in no cluster)
      uint16_t* queue = queues[tid >> 5] + (tid & 31);
#pragma unroll 1
      for (int r0 = 0; r0 < L; r0 += ROUND, h0 += ROUND) {
        if (r0) read();
        // What concerns these slices goes through a queue per lane: few of a warp's
        // lanes with something to count do not hold up the others token by token.
        int queued = 0;
#pragma unroll
        for (int u = 0; u < HISTORY_AHEAD; u++) {
          const uint32_t at = (uint32_t)token[u] - (uint32_t)base;  // (a token below 0: far above)
          if (at < range && ahead(u) < L - h0) queue[32 * queued++] = (uint16_t)(at | (ahead(u) < prompt - h0 ? 0x8000u : 0u));
        }
        const int most = __reduce_max_sync(0xFFFFFFFFu, queued);
        for (int i = 0; i < most; i++) {
          if (i >= queued) continue;
          const uint32_t e = queue[32 * i], at = e & 0x7FFF;
          if (CLUSTERS) {
            if (e >> 15)
              atomicOr(&shared[at], IN_PROMPT);
            else
              atomicAdd(&shared[at], 1u);
          } else if ((e >> 15 ? atomicOr(&words[at], IN_PROMPT) : atomicAdd(&words[at], 1u)) == 0) {
            list[atomicAdd(&listed, 1)] = (uint16_t)at;
          }
        }
      }
      if constexpr (CLUSTERS) {
        cluster_arrive();
        cluster_wait();
        const uint32_t mine = smem_u32(words);
        for (int i = tid; i < S; i += ADJUST_THREADS) {
          uint32_t w[C], sum = 0;
#pragma unroll
          for (int r = 0; r < C; r++)
            asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(w[r]) : "r"(dsmem_addr_u32(mine + i * 4, r)) : "memory");
#pragma unroll
          for (int r = 0; r < C; r++) sum = ((sum & ~IN_PROMPT) + (w[r] & ~IN_PROMPT)) | ((sum | w[r]) & IN_PROMPT);
          words[i] = sum;  // read by this block alone
          if (sum) list[atomicAdd(&listed, 1)] = (uint16_t)i;
        }
        cluster_arrive();  // waited for at the end: no block leaves while others read its words
      }
      __syncthreads();
    } else if (!clear()) {
      return;
    }
    if (a.n_bias) {
      for (int i0 = ADJUST_THREADS; i0 < a.n_bias; i0 += ADJUST_THREADS) {  // a longer list's
        const int i = i0 + tid;
        first_bias = i < a.n_bias ? a.bias_token[b * a.bias_stride + i] : -1;
        first_value = i < a.n_bias ? a.bias[b * a.bias_stride + i] : 0.f;
        __syncthreads();
        find_biases();
        __syncthreads();
        hold_biases();
      }
      if (!counts || a.n_bias > ADJUST_THREADS) __syncthreads();
      // A word names the first bias of its token; the others (few lists have any) are
      // added to that one, in order.
      constexpr uint32_t SLOT = 0x7FFu << 20;
      auto first_of = [&](int k) {  // whether bias k is its token's first
        const uint32_t word = words[bias_at[k]];
        if (slot_of(word) != (uint32_t)k + 1) return false;
        if (!(word & ~SLOT)) list[atomicAdd(&listed, 1)] = bias_at[k];
        return true;
      };
      auto name = [&](int k) {
        uint32_t* word = &words[bias_at[k]];
        for (uint32_t old = *word; !slot_of(old) || slot_of(old) > (uint32_t)k + 1;) {
          const uint32_t seen = atomicCAS(word, old, (old & ~SLOT) | (uint32_t)(k + 1) << 20);
          if (seen == old) break;
          old = seen;
        }
      };
      auto add_others = [&] {  // one warp
        for (int k0 = 0; k0 < held; k0 += 32) {
          const int k = k0 + tid, slot = k < held ? (int)slot_of(words[bias_at[k]]) : 0;
          uint32_t again = __ballot_sync(0xFFFFFFFFu, k < held && slot != k + 1);
          while (again) {
            if (tid == __ffs(again) - 1) bias[slot - 1] += bias[k];
            again &= again - 1;
            __syncwarp();
          }
        }
      };
      if (a.n_bias <= 32) {  // the first warp's
        if (tid < 32) {
          if (tid < held) name(tid);
          __syncwarp();
          if (__any_sync(0xFFFFFFFFu, tid < held && !first_of(tid))) add_others();
        }
      } else {
        for (int k = tid; k < held; k += ADJUST_THREADS) name(k);
        __syncthreads();
        bool others = false;
        for (int k = tid; k < held; k += ADJUST_THREADS) others |= !first_of(k);
        if (__syncthreads_or(others) && tid < 32) add_others();
      }
    }
    if (a.n_bias || DRAFTS)
      any_draft = __syncthreads_or(DRAFTS && tid < p.T && draft[tid] >= 0 && (uint32_t)(draft[tid] - v0) < (uint32_t)n);
    fixes = counts || a.n_bias ? listed * rows : 0;
  } else {
    copy();
  }
  Penalties value = {1.f, 0.f, 0.f};
  if (a.repetition) value.r = a.repetition[b];
  if (!(value.r > 0.f)) value.r = 1.f;
  if (a.presence) value.p = a.presence[b];
  if (a.frequency) value.f = a.frequency[b];

  // Tokens of the tree's rows: a row's path counts its own, on top of the history.
  // Their values are formed before any changed one is written, as out may be the logits.
  float path_value[DRAFTS ? MAX_PAIRS : 1];
  uint32_t path_here = 0;
  if (DRAFTS && any_draft) {
#pragma unroll
    for (int k = 0; k < MAX_PAIRS; k++) {
      const int pair = tid + k * ADJUST_THREADS, t = pair / p.T, j = pair % p.T;
      if (t >= p.T || !(tree[t] >> j & 1) || draft[j] < v0 || draft[j] >= v0 + n) continue;
      uint32_t more = 0;
      bool first = true;
      for (int i = 0; i < p.T; i++)
        if (tree[t] >> i & 1 && draft[i] == draft[j]) {
          more++;
          if (i < j) first = false;
        }
      const int at = draft[j] - v0;
      if (!first || (a.allowed && !(allowed_bits(t, at, at + 1) & 1))) continue;
      path_value[k] = value(to_float(static_cast<const T*>(p.logits)[(row0 + t) * p.ld + draft[j]]), words[at], more, bias);
      path_here |= 1u << k;
    }
  }

  // Changed logits, FIXES_AHEAD of them at once: their logits and whether they are
  // allowed, then their values.  (The copy has left allowed logits as they were,
  // also in place.)
  float y[FIXES_AHEAD];
  uint32_t stands = 0;
  const uint32_t per_row = fixes ? (uint32_t)listed : 1u, per_row_inverse = ONE ? 0u : 0xFFFFFFFFu / per_row + 1;
  auto row_of = [&](int i) {  // i / per_row
    if (ONE) return 0;
    if (per_row == 1) return i;
    const int t = (int)__umulhi((uint32_t)i, per_row_inverse);  // or one more, far out
    return t * (int)per_row > i ? t - 1 : t;
  };
  auto fetch = [&](int i0) {
    stands = 0;
#pragma unroll
    for (int k = 0; k < FIXES_AHEAD; k++) {
      const int i = i0 + k * ADJUST_THREADS;
      if (i >= fixes) continue;
      const int t = row_of(i), at = list[i - t * (int)per_row];
      y[k] = to_float(static_cast<const T*>(p.logits)[(row0 + t) * p.ld + v0 + at]);
      stands |= (a.allowed ? allowed_bits(t, at, at + 1) & 1 : 1u) << k;
    }
  };
  auto settle = [&](int i0) {
#pragma unroll
    for (int k = 0; k < FIXES_AHEAD; k++) {
      const int i = i0 + k * ADJUST_THREADS;
      if (!(stands >> k & 1)) continue;
      const int t = row_of(i), at = list[i - t * (int)per_row];
      static_cast<T*>(p.out)[(row0 + t) * p.out_ld + v0 + at] = from_float<T>(value(y[k], words[at], 0, bias));
    }
  };
  // ---- what changes
  if (DRAFTS && any_draft && p.in_place) __syncthreads();
#pragma unroll 1
  for (int i0 = tid; i0 < fixes; i0 += FIXES_AHEAD * ADJUST_THREADS) {
    fetch(i0);
    settle(i0);
  }
  if (DRAFTS && any_draft) {
    __syncthreads();
#pragma unroll
    for (int k = 0; k < MAX_PAIRS; k++) {
      const int pair = tid + k * ADJUST_THREADS, t = pair / p.T, j = pair % p.T;
      if (path_here >> k & 1) static_cast<T*>(p.out)[(row0 + t) * p.out_ld + draft[j]] = from_float<T>(path_value[k]);
    }
  }
  if constexpr (CLUSTERS) cluster_wait();
}

struct AdjustDevice {
  std::once_flag once;
  qlin_status ready = QLIN_ERR_CUDA;
  int sms = 0;
};
AdjustDevice g_adjust[64];

constexpr int64_t adjust_smem(int64_t slice, int cluster) { return slice * (4 * cluster + 2); }

template <typename T, bool CLUSTERS>
const void* adjust_fn_t(Rows kind) {
  return kind == Rows::ONE       ? reinterpret_cast<const void*>(qlin_adjust_kernel<T, CLUSTERS, Rows::ONE>)
         : kind == Rows::SEVERAL ? reinterpret_cast<const void*>(qlin_adjust_kernel<T, CLUSTERS, Rows::SEVERAL>)
                                 : reinterpret_cast<const void*>(qlin_adjust_kernel<T, CLUSTERS, Rows::DRAFTED>);
}
const void* adjust_fn(int dtype, bool clusters, Rows kind) {
  if (dtype == QLIN_F32) return clusters ? adjust_fn_t<float, true>(kind) : adjust_fn_t<float, false>(kind);
  return clusters ? adjust_fn_t<__nv_bfloat16, true>(kind) : adjust_fn_t<__nv_bfloat16, false>(kind);
}

qlin_status adjust_setup(int* sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return status_of(e);
  if (dev < 0 || dev >= 64) return QLIN_ERR_CUDA;
  AdjustDevice& d = g_adjust[dev];
  std::call_once(d.once, [&d, dev] {
    cudaError_t e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
    for (int dtype : {QLIN_F32, QLIN_BF16})
      for (bool clusters : {false, true})
        for (Rows kind : {Rows::ONE, Rows::SEVERAL, Rows::DRAFTED})
          if (e == cudaSuccess)
            e = cudaFuncSetAttribute(adjust_fn(dtype, clusters, kind), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)(clusters ? adjust_smem(CLUSTER_SLICE, CLUSTER) : adjust_smem(AHEAD * ADJUST_THREADS * 8, 1)));
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
  if (V > QLIN_SAMPLE_MAX_V || B > QLIN_MAX_SEQUENCES || T > 65535 * ROWS || (int64_t)B * T > (1 << 24) || a.L > QLIN_MAX_HISTORY ||
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
  const Rows kind = a.draft ? Rows::DRAFTED : T > 1 ? Rows::SEVERAL : Rows::ONE;
  p.history_vectors = a.history && is_aligned(a.history, 16) && a.L % 4 == 0 && (B == 1 || a.history_stride % 4 == 0);
  // A thread's vectors of a block: AHEAD, or fewer where that leaves SMs idle; then
  // as many as make the blocks fill whole rounds of the SMs.  Rows off the 16-byte
  // grid take one vector more than their slice has.
  const int64_t vec = 16 / size, rows = T < ROWS ? T : ROWS, groups = B * ((T + ROWS - 1) / ROWS);
  const int64_t spare = is_aligned(logits, 16) && (M == 1 || ld % vec == 0) ? 0 : 1;
  const int64_t round = BLOCKS * sms;
  int64_t vectors = AHEAD * ADJUST_THREADS / rows;  // of a row, at most
  auto slices_of = [&](int64_t vectors) { return (V + (vectors - spare) * vec - 1) / ((vectors - spare) * vec); };
  // Clusters where their smaller slices still make one round of blocks (8 rows of
  // 131071 and 20011 tokens 12.8 us, 15.6 without), not where they make several (64
  // rows of 131071 and 8000 tokens 73 us, 30 without), and again where the history
  // is so long that reading it in each block costs more than the rounds (64 rows of
  // 32000 and 60000 tokens 28 us, 42 without).  That border lies at one length for
  // all vocabularies, and too low for large ones: 64 rows of 131071 and 50000 tokens
  // take 83 us, 74 without.  The length is the history's width, as those in use are
  // known on the device alone: 8000 tokens in one of 40000 take those rows 71 us, 29
  // in one of 8000.
  const int64_t fewer = std::min(vectors, CLUSTER_SLICE / vec + spare);
  const int64_t in_clusters = (slices_of(fewer) + CLUSTER - 1) / CLUSTER * CLUSTER;
  const bool clusters = a.history && V > 4096 && a.L > (in_clusters * groups <= round ? LONG_HISTORY : VERY_LONG_HISTORY);
  if (clusters) vectors = fewer;
  int64_t slices = clusters ? in_clusters : slices_of(vectors);
  const int64_t rounds = (slices * groups + round - 1) / round;
  slices = rounds * round / groups;  // at least as many
  if (clusters) slices = slices / CLUSTER * CLUSTER;
  const int64_t least = (V + slices * vec - 1) / (slices * vec) + spare;
  if (vectors > least) vectors = least;
  if (vectors < 128) vectors = 128;
  const int64_t slice = (vectors - spare) * vec;
  slices = (V + slice - 1) / slice;
  if (clusters) slices = (slices + CLUSTER - 1) / CLUSTER * CLUSTER;
  p.aligned = !spare && is_aligned(out, 16) && (M == 1 || out_ld % vec == 0);
  p.slice = (int)slice;
  p.vectors = (int)vectors;
  p.vectors_inverse = (uint32_t)(((1ull << 32) + vectors - 1) / vectors);
  void* args[] = {&p};
  return launch_step(adjust_fn(dtype, clusters, kind), dim3((unsigned)slices, (unsigned)B, (unsigned)((T + ROWS - 1) / ROWS)),
                     dim3(ADJUST_THREADS, 1, 1), (size_t)adjust_smem(slice, clusters ? CLUSTER : 1),
                     static_cast<cudaStream_t>(stream), args, (flags & QLIN_FLAG_PDL) != 0, clusters ? CLUSTER : 1);
}
