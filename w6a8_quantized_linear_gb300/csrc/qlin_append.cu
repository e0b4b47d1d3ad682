// qlin_kv_append and qlin_kv_keep: a step's projected rows into the paged
// cache, and an accepted path moved up behind the committed tokens.
#include <cmath>

#include "qlin_ptx.cuh"
#include "qlin_step.h"

namespace qlin {
namespace {

constexpr int APPEND_THREADS = 128;

struct AppendParams {
  qlin_kv_cache cache;
  qlin_kv_step step;
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride, q_out_stride;
  void* q_out;
  const float *q_gamma, *k_gamma;
  const uint64_t* turns;
  const int32_t* position;  // a row's positions, `position_stride` apart between rows, or none: len + depth
  int64_t position_stride;
  uint64_t axis[4];         // which of a row's positions turns pair i: bits 2 (i % 32) of word i / 32, a word per warp
  uint32_t* status;
  float eps;
  int Hq, n_turns, pairs;
  int heads;  // head rows of a token: of q, k and v
  int heads_per_block;
};

// A thread's two runs of R elements of a head, as they were loaded.
template <typename SRC, int R>
struct Raw;
template <>
struct Raw<float, 4> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p, int half) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + half);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
};
template <int R>
struct Raw<__nv_bfloat16, R> {
  uint32_t w[R];  // two elements each
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int half) {
    if constexpr (R == 4) {
      *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(p);
      *reinterpret_cast<uint2*>(w + 2) = *reinterpret_cast<const uint2*>(p + half);
    } else {
      *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(p);
      *reinterpret_cast<uint4*>(w + 4) = *reinterpret_cast<const uint4*>(p + half);
    }
  }
  __device__ __forceinline__ void get(float (&x)[2 * R]) const {
#pragma unroll
    for (int e = 0; e < R; e++) {
      const float2 f = unpack2(w[e], __nv_bfloat16());
      x[2 * e] = f.x, x[2 * e + 1] = f.y;
    }
  }
};
template <int R, typename DST>
__device__ __forceinline__ void store_run(const float* x, DST* p) {
  const uint2 lo = make_uint2(pack2(x[0], x[1], DST()), pack2(x[2], x[3], DST()));
  if constexpr (R == 4)
    *reinterpret_cast<uint2*>(p) = lo;
  else
    *reinterpret_cast<uint4*>(p) = make_uint4(lo.x, lo.y, pack2(x[4], x[5], DST()), pack2(x[6], x[7], DST()));
}

// One block per token row and run of heads; D / (2 R) lanes per head, so that a
// warp's instructions work on up to eight heads, and one to four passes' loads
// in flight.  Lane l of a head holds elements R l .. R l + R - 1 of each half, so that
// where a whole head turns, both of a pair are the lane's own.
//   x' = x gamma / sqrt(mean(x^2) + eps);  (a, b) -> (a cos - b sin, b cos + a sin)
// The angle is pos * turns[i] mod 1, exact in 64-bit integers whatever the
// position, so only its last conversion to fp32 rounds; pos is the row's place, or
// its given position on the axis of pair i (two bits per pair, a word per warp, so
// that a thread reads its own with the rows).  Bound by the bytes of
// the rows for a prompt in fp32 (6 per element), by the launch for a step; in bf16
// by no unit alone (issue 0.67 of the cycles, DRAM 29 %, warps 43 %): a block's start
// (length, page, angles, a barrier) stands before each row's work.
// Measured, 4001 rows of 64 heads of 128: fp32 34.2 us (197 MB, 5.7 TB/s, 0.85
// of the measured copy), bf16 26.1 us (131 MB).  A warp per head with four elements
// a lane issued three times the instructions and was bound by them (48 us).  At
// positions of three axes: 4098 rows of 64 heads of 128 in fp32 35.1 us (0.85 of the
// copy), 2411 of 32 heads of 256 in bf16 17.5 us (79 MB).
// R = 8 where a bf16 prompt's rows fill a pass of blocks: twice the elements share a
// lane's addresses, shuffles and root (30.4 and 21.9 us with R = 4).  One pass in
// flight and eight blocks per SM then do better than two and seven (26.3 and 19.7).
template <typename SRC, typename DST, int D, int R>
__global__ void __launch_bounds__(APPEND_THREADS, R == 8 ? 8 : 7) qlin_append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int LANES = D / (2 * R), PASS = APPEND_THREADS / LANES;  // lanes of a head, heads of a pass
  constexpr int AHEAD = R == 8 ? 1 : sizeof(SRC) == 4 ? 2 : 4;  // passes in flight: 64 bytes a thread, or 32
  constexpr int H = D / 2;
  __shared__ float2 cs[D / 2];                  // cos, sin of this row's angles
  __shared__ __align__(16) float gamma[2][D];   // of q, of k
  __shared__ float rows[PASS][D];
  const int row = blockIdx.x, b = row / p.step.T, t = row - b * p.step.T;
  const int at0 = threadIdx.x % LANES * R, slot = threadIdx.x / LANES;  // this thread's elements, its head of a pass
  pdl_wait();
  pdl_launch_dependents();
  // everything that is read goes out before anything is waited for
  const int h1 = min((int)(blockIdx.y + 1) * p.heads_per_block, p.heads);
  const int h = blockIdx.y * p.heads_per_block + slot;
  // the heads of a token: of q, then of k, then of v
  const int v0 = p.Hq + p.cache.heads;
  const SRC* qs = static_cast<const SRC*>(p.q) + row * p.q_stride + at0;
  const SRC* ks = static_cast<const SRC*>(p.k) + (row * p.k_stride - (int64_t)p.Hq * D) + at0;
  const SRC* vs = static_cast<const SRC*>(p.v) + (row * p.v_stride - (int64_t)v0 * D) + at0;
  auto load = [&](Raw<SRC, R>& x, int head) { x.load((head < p.Hq ? qs : head < v0 ? ks : vs) + head * D, H); };
  Raw<SRC, R> x[AHEAD];
#pragma unroll
  for (int u = 0; u < AHEAD; u++)
    if (h + u * PASS < h1) load(x[u], h + u * PASS);
  const uint64_t turn = threadIdx.x < p.n_turns ? p.turns[threadIdx.x] : 0;
  for (int i = threadIdx.x; i < D; i += APPEND_THREADS) {
    gamma[0][i] = p.q_gamma ? p.q_gamma[i] : 1.f;
    gamma[1][i] = p.k_gamma ? p.k_gamma[i] : 1.f;
  }
  const int len = p.step.len[b], used = step_rows(p.step, b);
  int64_t pos;
  if (p.position)
    pos = threadIdx.x < p.n_turns
              ? p.position[row * p.position_stride + (p.axis[threadIdx.x / 32] >> 2 * (threadIdx.x % 32) & 3)] : 0;
  else
    pos = (int64_t)len + (p.step.depth ? p.step.depth[b * p.step.tree_stride + t] : t);
  if (len < 0 || t >= used) return;
  const int n = p.n_turns;
  static_assert(APPEND_THREADS >= D / 2, "a thread per angle");
  if (threadIdx.x < n) {
    const int64_t angle = (int64_t)((uint64_t)pos * turn);  // in [-1/2, 1/2) turns of 2^64
    float s, c;
    sincospif((float)(int32_t)(angle >> 32) * 0x1p-31f, &s, &c);
    cs[threadIdx.x] = make_float2(c, s);
  }
  const int64_t at = p.k ? token_offset(p.cache, p.step, b, (int64_t)len + t) : 0;
  if (at < 0 && threadIdx.x == 0) report(p.status, QLIN_ERR_BAD_INDEX);
  __syncthreads();
  // How a head turns: not at all; pairs, or whole halves, within the lane;
  // a power of two of whole lanes, with lane ^ flip (or, of half a lane, within
  // it); any other, through shared memory.  The lane's cosines and sines are the
  // same for all heads.
  const bool across = !p.pairs && n && n < H && n % 4 == 0 && (n & (n - 1)) == 0 && 2 * n <= H;
  const bool near = R == 8 && across && n == 4;
  const int flip = across && !near ? n / R : 0;
  const bool own = !p.pairs && n == H;
  float tc[R], ts[R];  // pairs: of the even elements of each half; else of the first half's (across: signed by its side)
#pragma unroll
  for (int e = 0; e < R; e++) {
    int i = at0 + e;
    if (p.pairs) i = (e < R / 2 ? at0 + 2 * e : H + at0 + 2 * (e - R / 2)) / 2;
    const bool second = across && i >= n;
    if (second) i -= n;
    const float2 w = i < n ? cs[i] : make_float2(1.f, 0.f);
    tc[e] = w.x;
    ts[e] = across && !second ? -w.y : w.y;
  }
  DST* const qd = static_cast<DST*>(p.q_out) + row * p.q_out_stride + at0;
  auto finish = [&](float (&x)[2 * R], int head) {
    const bool is_q = head < p.Hq, is_v = head >= v0, here = head < h1;
    if (__any_sync(0xFFFFFFFFu, here && !is_v)) {  // all lanes: the warp's heads may differ in kind
      if (p.q_gamma || p.k_gamma) {
        // (four elements of each half at a time, and those added last: one order of
        // sums whatever a lane holds)
        float part[R / 4];
#pragma unroll
        for (int k = 0; k < R / 4; k++) {
          part[k] = 0.f;
#pragma unroll
          for (int e = 0; e < 8; e++) {
            const float y = x[e % 4 + 4 * k + e / 4 * R];
            part[k] = fmaf(y, y, part[k]);
          }
        }
#pragma unroll
        for (int o = LANES / 2; o; o >>= 1)
#pragma unroll
          for (int k = 0; k < R / 4; k++) part[k] += __shfl_xor_sync(0xFFFFFFFFu, part[k], o);
        const float ss = R == 4 ? part[0] : part[0] + part[R / 4 - 1];
        const float a = ss * (1.0f / D) + p.eps;
        float r = rsqrtf(a);  // and a Newton step, to one ulp (a = 0 or infinite: as it is)
        const float d = fmaf(-a * r, r, 1.f);
        if (fabsf(d) < 1.f) r = fmaf(0.5f * r, d, r);
        if ((is_q ? p.q_gamma : p.k_gamma) && !is_v) {
          const float* g = gamma[is_q ? 0 : 1] + at0;
#pragma unroll
          for (int k = 0; k < R; k += 4) {
            const float4 g0 = *reinterpret_cast<const float4*>(g + k), g1 = *reinterpret_cast<const float4*>(g + H + k);
            x[k] *= r * g0.x, x[k + 1] *= r * g0.y, x[k + 2] *= r * g0.z, x[k + 3] *= r * g0.w;
            x[R + k] *= r * g1.x, x[R + k + 1] *= r * g1.y, x[R + k + 2] *= r * g1.z, x[R + k + 3] *= r * g1.w;
          }
        }
      }
      if (p.pairs) {
#pragma unroll
        for (int e = 0; e < R; e++) {
          const int i = e < R / 2 ? 2 * e : R + 2 * (e - R / 2);
          const float u = x[i], w = x[i + 1];
          if ((e < R / 2 ? at0 + 2 * e : H + at0 + 2 * (e - R / 2)) < 2 * n && !is_v) {
            x[i] = u * tc[e] - w * ts[e];
            x[i + 1] = w * tc[e] + u * ts[e];
          }
        }
      } else if (own) {
        if (!is_v)
#pragma unroll
          for (int e = 0; e < R; e++) {
            const float u = x[e], w = x[R + e];
            x[e] = u * tc[e] - w * ts[e];
            x[R + e] = w * tc[e] + u * ts[e];
          }
      } else if (flip) {
#pragma unroll
        for (int e = 0; e < R; e++) {
          const float other = __shfl_xor_sync(0xFFFFFFFFu, x[e], flip);
          if (at0 < 2 * n && !is_v) x[e] = x[e] * tc[e] + other * ts[e];
        }
      } else if (near) {
        if constexpr (R == 8) {
          if (at0 == 0 && !is_v)
#pragma unroll
            for (int e = 0; e < 4; e++) {
              const float u = x[e], w = x[e + 4];
              x[e] = u * tc[e] + w * ts[e];
              x[e + 4] = w * tc[e + 4] + u * ts[e + 4];
            }
        }
      } else if (n) {
        float* mine = rows[slot];
#pragma unroll
        for (int e = 0; e < 2 * R; e++) mine[at0 + e % R + e / R * H] = x[e];
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 2 * R; e++) {
          const int i = at0 + e % R + e / R * H;
          if (i < 2 * n && !is_v) {
            const float2 w = cs[i >= n ? i - n : i];
            x[e] = i >= n ? x[e] * w.x + mine[i - n] * w.y : x[e] * w.x - mine[i + n] * w.y;
          }
        }
        __syncwarp();
      }
    }
    if (!here) return;
    if (is_q) {
      store_run<R>(x, qd + head * D);
      store_run<R>(x + R, qd + head * D + H);
    } else if (at >= 0) {
      DST* dst = static_cast<DST*>(is_v ? p.cache.v : p.cache.k) + at + (head - (is_v ? v0 : p.Hq)) * p.cache.head_stride + at0;
      store_run<R>(x, dst);
      store_run<R>(x + R, dst + H);
    }
  };
  const int warp_first = h - slot + (int)(threadIdx.x & ~31u) / LANES;  // the same in all lanes of a warp
  for (int off = 0; warp_first + off < h1; off += AHEAD * PASS) {
#pragma unroll
    for (int u = 0; u < AHEAD; u++) {
      const int head = h + off + u * PASS;
      if (warp_first + off + u * PASS >= h1) break;
      float now[2 * R];
      x[u].get(now);
      if (head + AHEAD * PASS < h1) load(x[u], head + AHEAD * PASS);
      finish(now, head);
    }
  }
}

template <typename SRC, typename DST, int R>
const void* append_fn_d(int width) {
  return width == 64    ? reinterpret_cast<const void*>(qlin_append_kernel<SRC, DST, 64, R>)
         : width == 128 ? reinterpret_cast<const void*>(qlin_append_kernel<SRC, DST, 128, R>)
                        : reinterpret_cast<const void*>(qlin_append_kernel<SRC, DST, 256, R>);
}
const void* append_fn(int src, int dst, int width, int run) {
  if (src == QLIN_F32)
    return dst == QLIN_BF16 ? append_fn_d<float, __nv_bfloat16, 4>(width) : append_fn_d<float, __half, 4>(width);
  if (run == 4)
    return dst == QLIN_BF16 ? append_fn_d<__nv_bfloat16, __nv_bfloat16, 4>(width)
                            : append_fn_d<__nv_bfloat16, __half, 4>(width);
  return dst == QLIN_BF16 ? append_fn_d<__nv_bfloat16, __nv_bfloat16, 8>(width) : append_fn_d<__nv_bfloat16, __half, 8>(width);
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

static qlin_status append(const qlin_kv_cache* cache, const qlin_kv_step* step, int Hq, int src, const void* q,
                          int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                          const float* q_gamma, const float* k_gamma, float eps, const uint64_t* turns, int n_turns,
                          int pairs, const int32_t* position, int64_t position_stride, int axes, const uint8_t* axis,
                          void* q_out, int64_t q_out_stride, void* ws, size_t ws_bytes, unsigned flags, void* stream) {
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
  if (position) {
    if (axes < 1 || axes > QLIN_MAX_AXES || !is_aligned(position, 4) || position_stride < axes ||
        (axes > 1 && n_turns && !axis))
      return QLIN_ERR_INVALID_ARG;
    for (int i = 0; axis && i < n_turns; i++)
      if (axis[i] >= axes) return QLIN_ERR_INVALID_ARG;
  }
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
  if (q) {  // a row of q_out is written while other heads of q, k and v are still to be read
    const int64_t n = (int64_t)step->B * step->T, kv = cache->heads * D;
    const bool in_place = q_out == q && size == 2 && q_out_stride == q_stride;  // a thread writes what it alone read
    if ((!in_place && rows_overlap(q_out, q_out_stride * 2, Hq * D * 2, q, q_stride * size, Hq * D * size, n)) ||
        rows_overlap(q_out, q_out_stride * 2, Hq * D * 2, k, k_stride * size, kv * size, n) ||
        rows_overlap(q_out, q_out_stride * 2, Hq * D * 2, v, v_stride * size, kv * size, n))
      return QLIN_ERR_INVALID_ARG;
    if (position && rows_overlap(q_out, q_out_stride * 2, Hq * D * 2, position, position_stride * 4, axes * 4, n))
      return QLIN_ERR_INVALID_ARG;
  }
  AppendParams p = {};
  p.cache = *cache;
  p.step = *step;
  p.q = q, p.k = k, p.v = v;
  p.q_stride = q_stride, p.k_stride = k_stride, p.v_stride = v_stride, p.q_out_stride = q_out_stride;
  p.q_out = q_out;
  p.q_gamma = q_gamma, p.k_gamma = k_gamma;
  p.turns = turns;
  p.position = position;
  p.position_stride = position_stride;
  for (int i = 0; position && axis && i < n_turns; i++) p.axis[i / 32] |= (uint64_t)axis[i] << 2 * (i % 32);
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
  // eight elements to a run where that leaves no lanes idle, and there is more than a step's rows
  const int run = src == QLIN_BF16 && rows >= 64 && p.heads >= APPEND_THREADS / (D / 16) ? 8 : 4;
  const int64_t pass = APPEND_THREADS / (D / (2 * run));
  per = (per + pass - 1) / pass * pass;
  p.heads_per_block = (int)per;
  void* args[] = {&p};
  return launch_step(append_fn(src, cache->dtype, cache->width, run),
                     dim3((unsigned)rows, (unsigned)((p.heads + per - 1) / per), 1), dim3(APPEND_THREADS, 1, 1), 0,
                     static_cast<cudaStream_t>(stream), args, (flags & QLIN_FLAG_PDL) != 0);
}

qlin_status qlin_kv_append(const qlin_kv_cache* cache, const qlin_kv_step* step, int Hq, int src, const void* q,
                           int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                           const float* q_gamma, const float* k_gamma, float eps, const uint64_t* turns, int n_turns,
                           int pairs, void* q_out, int64_t q_out_stride, void* ws, size_t ws_bytes, unsigned flags,
                           void* stream) {
  return append(cache, step, Hq, src, q, q_stride, k, k_stride, v, v_stride, q_gamma, k_gamma, eps, turns, n_turns,
                pairs, nullptr, 0, 0, nullptr, q_out, q_out_stride, ws, ws_bytes, flags, stream);
}

qlin_status qlin_kv_append_at(const qlin_kv_cache* cache, const qlin_kv_step* step, int Hq, int src, const void* q,
                              int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                              const float* q_gamma, const float* k_gamma, float eps, const uint64_t* turns,
                              int n_turns, int pairs, const int32_t* position, int64_t position_stride, int axes,
                              const uint8_t* axis, void* q_out, int64_t q_out_stride, void* ws, size_t ws_bytes,
                              unsigned flags, void* stream) {
  if (!position) {  // but an empty step has none to give
    if (!step || (step->B != 0 && step->T != 0)) return QLIN_ERR_INVALID_ARG;
  }
  return append(cache, step, Hq, src, q, q_stride, k, k_stride, v, v_stride, q_gamma, k_gamma, eps, turns, n_turns,
                pairs, position, position_stride, axes, axis, q_out, q_out_stride, ws, ws_bytes, flags, stream);
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
