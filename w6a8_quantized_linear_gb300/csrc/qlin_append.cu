// qlin_kv_append and qlin_kv_keep: a step's projected rows into the paged
// cache, and an accepted path moved up behind the committed tokens.
#include <cmath>

#include "qlin_ptx.cuh"
#include "qlin_step.h"

namespace qlin {
namespace {

constexpr int APPEND_WARPS = 8;

struct AppendParams {
  qlin_kv_cache cache;
  qlin_kv_step step;
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride, q_out_stride;
  void* q_out;
  const float *q_gamma, *k_gamma;
  const uint64_t* turns;
  uint32_t* status;
  float eps;
  int Hq, n_turns, pairs;
  int heads;  // head rows of a token: of q, k and v
  int heads_per_block;
};

// A head row of D elements on a warp: NC chunks of E consecutive elements a
// lane (chunk c covers elements c * 32 * E ..), so that each load and store of
// a warp is one contiguous run.
template <int D>
struct HeadRow {
  static constexpr int E = D >= 128 ? 4 : 2;
  static constexpr int NC = D / (32 * E);
  float x[NC][E];
};

template <int D>
__device__ __forceinline__ void load_row(HeadRow<D>& r, const float* p, int lane) {
#pragma unroll
  for (int c = 0; c < HeadRow<D>::NC; c++) {
    const float* s = p + (c * 32 + lane) * HeadRow<D>::E;
    if constexpr (HeadRow<D>::E == 4) {
      const float4 f = *reinterpret_cast<const float4*>(s);
      r.x[c][0] = f.x, r.x[c][1] = f.y, r.x[c][2] = f.z, r.x[c][3] = f.w;
    } else {
      const float2 f = *reinterpret_cast<const float2*>(s);
      r.x[c][0] = f.x, r.x[c][1] = f.y;
    }
  }
}
template <int D>
__device__ __forceinline__ void load_row(HeadRow<D>& r, const __nv_bfloat16* p, int lane) {
#pragma unroll
  for (int c = 0; c < HeadRow<D>::NC; c++) {
    const __nv_bfloat16* s = p + (c * 32 + lane) * HeadRow<D>::E;
#pragma unroll
    for (int e = 0; e < HeadRow<D>::E; e += 2) {
      const float2 f = unpack2(*reinterpret_cast<const uint32_t*>(s + e), __nv_bfloat16());
      r.x[c][e] = f.x, r.x[c][e + 1] = f.y;
    }
  }
}
template <int D, typename DST>
__device__ __forceinline__ void store_row(const HeadRow<D>& r, DST* p, int lane) {
#pragma unroll
  for (int c = 0; c < HeadRow<D>::NC; c++) {
    DST* s = p + (c * 32 + lane) * HeadRow<D>::E;
    if constexpr (HeadRow<D>::E == 4) {
      *reinterpret_cast<uint2*>(s) =
          make_uint2(pack2(r.x[c][0], r.x[c][1], DST()), pack2(r.x[c][2], r.x[c][3], DST()));
    } else {
      *reinterpret_cast<uint32_t*>(s) = pack2(r.x[c][0], r.x[c][1], DST());
    }
  }
}

// One block per token row and run of heads, one warp per head, two or four
// heads of a warp in flight.
//   x' = x gamma / sqrt(mean(x^2) + eps);  (a, b) -> (a cos - b sin, b cos + a sin)
// The angle is pos * turns[i] mod 1, exact in 64-bit integers whatever the
// position, so only its last conversion to fp32 rounds.  Bound by the bytes of
// the rows (6 or 4 per element) for a prompt, by the launch for a step.
template <typename SRC, typename DST, int D>
__global__ void __launch_bounds__(APPEND_WARPS * 32) qlin_append_kernel(const __grid_constant__ AppendParams p) {
  __shared__ float2 cs[D / 2];                     // cos, sin of this row's angles
  __shared__ float rows[APPEND_WARPS][D];
  constexpr int AHEAD = D == 256 ? 2 : 4;
  const int row = blockIdx.x, b = row / p.step.T, t = row - b * p.step.T;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_launch_dependents();
  const int len = p.step.len[b];
  if (len < 0 || t >= step_rows(p.step, b)) return;
  const int h0 = blockIdx.y * p.heads_per_block + warp;
  const int h1 = min((int)(blockIdx.y + 1) * p.heads_per_block, p.heads);
  // the heads of a token: of q, then of k, then of v
  auto load = [&](HeadRow<D>& x, int head) {
    const int hk = head - p.Hq;
    const SRC* src = hk < 0 ? static_cast<const SRC*>(p.q) + row * p.q_stride + (int64_t)head * D
                     : hk < p.cache.heads
                         ? static_cast<const SRC*>(p.k) + row * p.k_stride + (int64_t)hk * D
                         : static_cast<const SRC*>(p.v) + row * p.v_stride + (int64_t)(hk - p.cache.heads) * D;
    load_row<D>(x, src, lane);
  };
  HeadRow<D> x[AHEAD];
#pragma unroll
  for (int u = 0; u < AHEAD; u++)
    if (h0 + u * APPEND_WARPS < h1) load(x[u], h0 + u * APPEND_WARPS);
  const int depth = p.step.depth ? p.step.depth[b * p.step.tree_stride + t] : t;
  const int64_t pos = (int64_t)len + depth;
  for (int i = threadIdx.x; i < p.n_turns; i += APPEND_WARPS * 32) {
    const int64_t turn = (int64_t)((uint64_t)pos * p.turns[i]);  // in [-1/2, 1/2) turns of 2^64
    float s, c;
    sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &s, &c);
    cs[i] = make_float2(c, s);
  }
  const int64_t at = p.k ? token_offset(p.cache, p.step, b, (int64_t)len + t) : 0;
  if (at < 0 && threadIdx.x == 0) report(p.status, QLIN_ERR_BAD_INDEX);
  __syncthreads();
  auto finish = [&](HeadRow<D>& x, int head) {
    const int hk = head - p.Hq;
    const bool is_q = hk < 0, is_v = hk >= p.cache.heads;
    if (!is_v) {
      const float* gamma = is_q ? p.q_gamma : p.k_gamma;
      if (gamma) {
        HeadRow<D> g;
        load_row<D>(g, gamma, lane);
        float ss = 0.f;
#pragma unroll
        for (int c = 0; c < x.NC; c++)
#pragma unroll
          for (int e = 0; e < x.E; e++) ss = fmaf(x.x[c][e], x.x[c][e], ss);
#pragma unroll
        for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
        const float r = 1.0f / sqrtf(ss * (1.0f / D) + p.eps);
#pragma unroll
        for (int c = 0; c < x.NC; c++)
#pragma unroll
          for (int e = 0; e < x.E; e++) x.x[c][e] *= r * g.x[c][e];
      }
      if (p.n_turns) {
        float* mine = rows[warp];
        if (!p.pairs) {  // the other of a pair may be another lane's
#pragma unroll
          for (int c = 0; c < x.NC; c++)
#pragma unroll
            for (int e = 0; e < x.E; e++) mine[(c * 32 + lane) * x.E + e] = x.x[c][e];
          __syncwarp();
        }
#pragma unroll
        for (int c = 0; c < x.NC; c++)
#pragma unroll
          for (int e = 0; e < x.E; e += 2) {
            const int i = (c * 32 + lane) * x.E + e;
            if (i >= 2 * p.n_turns) continue;
            if (p.pairs) {
              const float2 w = cs[i >> 1];
              const float a = x.x[c][e], b2 = x.x[c][e + 1];
              x.x[c][e] = a * w.x - b2 * w.y;
              x.x[c][e + 1] = b2 * w.x + a * w.y;
            } else {
#pragma unroll
              for (int k = 0; k < 2; k++) {
                const bool second = i + k >= p.n_turns;
                if (i + k < 2 * p.n_turns) {
                  const float other = mine[second ? i + k - p.n_turns : i + k + p.n_turns];
                  const float2 w = cs[second ? i + k - p.n_turns : i + k];
                  x.x[c][e + k] = x.x[c][e + k] * w.x + (second ? other : -other) * w.y;
                }
              }
            }
          }
        __syncwarp();
      }
    }
    if (is_q) {
      store_row<D>(x, static_cast<DST*>(p.q_out) + row * p.q_out_stride + (int64_t)head * D, lane);
    } else if (at >= 0) {
      DST* dst = static_cast<DST*>(is_v ? p.cache.v : p.cache.k);
      store_row<D>(x, dst + at + (is_v ? hk - p.cache.heads : hk) * p.cache.head_stride, lane);
    }
  };
  for (int h = h0; h < h1; h += AHEAD * APPEND_WARPS) {
#pragma unroll
    for (int u = 0; u < AHEAD; u++) {
      const int head = h + u * APPEND_WARPS;
      if (head < h1) {
        HeadRow<D> now = x[u];
        if (head + AHEAD * APPEND_WARPS < h1) load(x[u], head + AHEAD * APPEND_WARPS);
        finish(now, head);
      }
    }
  }
}

template <typename SRC, typename DST>
const void* append_fn_d(int width) {
  return width == 64    ? reinterpret_cast<const void*>(qlin_append_kernel<SRC, DST, 64>)
         : width == 128 ? reinterpret_cast<const void*>(qlin_append_kernel<SRC, DST, 128>)
                        : reinterpret_cast<const void*>(qlin_append_kernel<SRC, DST, 256>);
}
const void* append_fn(int src, int dst, int width) {
  if (src == QLIN_F32)
    return dst == QLIN_BF16 ? append_fn_d<float, __nv_bfloat16>(width) : append_fn_d<float, __half>(width);
  return dst == QLIN_BF16 ? append_fn_d<__nv_bfloat16, __nv_bfloat16>(width)
                          : append_fn_d<__nv_bfloat16, __half>(width);
}

// ---- keep ----------------------------------------------------------------------

constexpr int KEEP_THREADS = 512;

struct KeepParams {
  qlin_kv_cache cache;
  qlin_kv_step step;
  const int32_t *keep, *n_keep;
  int64_t keep_stride;
  int32_t* len_out;
  uint32_t* status;
};

// One block per sequence.  A thread moves one 16-byte column of a (k or v,
// head) row through all kept rows, in order: the list increases, so place i
// (<= keep[i]) is never a row that a later one still reads.  len is read by
// this block alone and written behind its barrier, so it may be advanced in
// place.
__global__ void __launch_bounds__(KEEP_THREADS) qlin_keep_kernel(const __grid_constant__ KeepParams p) {
  __shared__ int64_t from[QLIN_MAX_TREE], to[QLIN_MAX_TREE];
  __shared__ int bad;
  const int b = blockIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  const int len = p.step.len[b];
  if (len < 0) return;
  const int rows = step_rows(p.step, b);
  int n = p.n_keep[b];
  if (threadIdx.x == 0) bad = n < 0 || n > rows;
  __syncthreads();
  if (!bad && threadIdx.x < n) {
    const int i = threadIdx.x;
    const int r = p.keep[b * p.keep_stride + i];
    const int before = i ? p.keep[b * p.keep_stride + i - 1] : -1;
    if (r <= before || r >= rows) {
      bad = 1;
    } else {
      from[i] = token_offset(p.cache, p.step, b, (int64_t)len + r);
      to[i] = token_offset(p.cache, p.step, b, (int64_t)len + i);
      if (from[i] < 0 || to[i] < 0) bad = 1;
    }
  }
  __syncthreads();
  if (bad) {
    if (threadIdx.x == 0) {
      report(p.status, QLIN_ERR_BAD_INDEX);
      if (p.len_out) p.len_out[b] = len;
    }
    return;
  }
  const int per_head = p.cache.width / 8;
  const int columns = 2 * p.cache.heads * per_head;
  for (int c = threadIdx.x; c < columns; c += KEEP_THREADS) {
    const int head = (c / per_head) % p.cache.heads;
    uint16_t* base = static_cast<uint16_t*>(c < columns / 2 ? p.cache.k : p.cache.v) + head * p.cache.head_stride +
                     (c % per_head) * 8;
    for (int i = 0; i < n; i += 4) {  // four rows in flight, all read before the first is written
      uint4 x[4];
#pragma unroll
      for (int j = 0; j < 4; j++)
        if (i + j < n) x[j] = *reinterpret_cast<const uint4*>(base + from[i + j]);
#pragma unroll
      for (int j = 0; j < 4; j++)
        if (i + j < n && to[i + j] != from[i + j]) *reinterpret_cast<uint4*>(base + to[i + j]) = x[j];
    }
  }
  if (threadIdx.x == 0 && p.len_out) p.len_out[b] = len + n;
}

}  // namespace
}  // namespace qlin

using namespace qlin;

extern "C" {

qlin_status qlin_rope_turns(const double* radians, int n, uint64_t* turns) {
  if (n < 0 || n > 128 || (n && (!radians || !turns))) return QLIN_ERR_INVALID_ARG;
  for (int i = 0; i < n; i++)
    if (!std::isfinite(radians[i])) return QLIN_ERR_INVALID_ARG;
  for (int i = 0; i < n; i++) {
    double f = radians[i] / 6.283185307179586476925;
    f -= std::floor(f);  // [0, 1]: 1 only where a tiny negative rounds up to it
    turns[i] = f >= 1.0 ? 0 : (uint64_t)std::ldexp(f, 64);
  }
  return QLIN_OK;
}

qlin_status qlin_kv_append(const qlin_kv_cache* cache, const qlin_kv_step* step, int Hq, int src, const void* q,
                           int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                           const float* q_gamma, const float* k_gamma, float eps, const uint64_t* turns, int n_turns,
                           int pairs, void* q_out, int64_t q_out_stride, void* ws, size_t ws_bytes, unsigned flags,
                           void* stream) {
  qlin_status st = check_cache(cache);
  if (st != QLIN_OK) return st;
  st = check_step(step, 0x7FFFFFFF);
  if (st != QLIN_OK) return st;
  if (flags & ~QLIN_FLAG_PDL) return QLIN_ERR_INVALID_ARG;
  if (src != QLIN_F32 && src != QLIN_BF16) return QLIN_ERR_INVALID_ARG;
  if (Hq < 0 || n_turns < 0 || 2 * (int64_t)n_turns > cache->width || (pairs != 0 && pairs != 1))
    return QLIN_ERR_INVALID_ARG;
  if (Hq > 16384) return QLIN_ERR_UNSUPPORTED;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return QLIN_ERR_INVALID_ARG;
  if ((q_gamma && !is_aligned(q_gamma, 16)) || (k_gamma && !is_aligned(k_gamma, 16))) return QLIN_ERR_INVALID_ARG;
  if (n_turns && (!turns || !is_aligned(turns, 8))) return QLIN_ERR_INVALID_ARG;
  if ((k == nullptr) != (v == nullptr)) return QLIN_ERR_INVALID_ARG;
  st = check_status_ws(ws, ws_bytes);
  if (st != QLIN_OK) return st;
  if (step->B == 0 || step->T == 0) return QLIN_OK;
  const int64_t size = src == QLIN_F32 ? 4 : 2, D = cache->width;
  if (q) {
    if (Hq < 1 || !rows_ok(q, q_stride, Hq * D, size) || !rows_ok(q_out, q_out_stride, Hq * D, 2))
      return QLIN_ERR_INVALID_ARG;
  }
  if (k && (!rows_ok(k, k_stride, cache->heads * D, size) || !rows_ok(v, v_stride, cache->heads * D, size)))
    return QLIN_ERR_INVALID_ARG;
  if (!q && !k) return QLIN_OK;
  AppendParams p = {};
  p.cache = *cache;
  p.step = *step;
  p.q = q, p.k = k, p.v = v;
  p.q_stride = q_stride, p.k_stride = k_stride, p.v_stride = v_stride, p.q_out_stride = q_out_stride;
  p.q_out = q_out;
  p.q_gamma = q_gamma, p.k_gamma = k_gamma;
  p.turns = turns;
  p.status = static_cast<uint32_t*>(ws);
  p.eps = eps;
  p.Hq = q ? Hq : 0;
  p.n_turns = n_turns;
  p.pairs = pairs;
  p.heads = p.Hq + (k ? 2 * cache->heads : 0);
  const int64_t rows = (int64_t)step->B * step->T;
  // a few blocks per SM where the step has that many heads, a whole row per block beyond
  const int64_t want = (1216 + rows - 1) / rows;
  int64_t per = (p.heads + want - 1) / want;
  per = (per + APPEND_WARPS - 1) / APPEND_WARPS * APPEND_WARPS;
  p.heads_per_block = (int)per;
  void* args[] = {&p};
  return launch_step(append_fn(src, cache->dtype, cache->width),
                     dim3((unsigned)rows, (unsigned)((p.heads + per - 1) / per), 1), dim3(APPEND_WARPS * 32, 1, 1), 0,
                     static_cast<cudaStream_t>(stream), args, (flags & QLIN_FLAG_PDL) != 0);
}

qlin_status qlin_kv_keep(const qlin_kv_cache* cache, const qlin_kv_step* step, const int32_t* keep,
                         int64_t keep_stride, const int32_t* n_keep, int32_t* len_out, void* ws, size_t ws_bytes,
                         unsigned flags, void* stream) {
  qlin_status st = check_cache(cache);
  if (st != QLIN_OK) return st;
  st = check_step(step, QLIN_MAX_TREE);
  if (st != QLIN_OK) return st;
  if (flags & ~QLIN_FLAG_PDL) return QLIN_ERR_INVALID_ARG;
  st = check_status_ws(ws, ws_bytes);
  if (st != QLIN_OK) return st;
  if (step->B == 0 || step->T == 0) return QLIN_OK;
  if (!keep || !is_aligned(keep, 4) || !n_keep || !is_aligned(n_keep, 4) || !is_aligned(len_out, 4) ||
      keep_stride < step->T)
    return QLIN_ERR_INVALID_ARG;
  KeepParams p = {*cache, *step, keep, n_keep, keep_stride, len_out, static_cast<uint32_t*>(ws)};
  void* args[] = {&p};
  return launch_step(reinterpret_cast<const void*>(qlin_keep_kernel), dim3((unsigned)step->B, 1, 1),
                     dim3(KEEP_THREADS, 1, 1), 0, static_cast<cudaStream_t>(stream), args,
                     (flags & QLIN_FLAG_PDL) != 0);
}

}  // extern "C"
