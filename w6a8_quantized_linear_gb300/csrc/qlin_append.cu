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
  uint32_t* status;
  float eps;
  int Hq, n_turns, pairs;
  int heads;  // head rows of a token: of q, k and v
  int heads_per_block;
};

// A thread's two runs of four elements of a head, as they were loaded.
template <typename SRC>
struct Raw;
template <>
struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p, int half) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + half);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
};
template <>
struct Raw<__nv_bfloat16> {
  uint2 a, b;
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int half) {
    a = *reinterpret_cast<const uint2*>(p);
    b = *reinterpret_cast<const uint2*>(p + half);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
    for (int e = 0; e < 4; e++) {
      const float2 f = unpack2(w[e], __nv_bfloat16());
      x[2 * e] = f.x, x[2 * e + 1] = f.y;
    }
  }
};
template <typename DST>
__device__ __forceinline__ void store4(const float* x, DST* p) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack2(x[0], x[1], DST()), pack2(x[2], x[3], DST()));
}

// One block per token row and run of heads; D / 8 lanes per head, so that a
// warp's instructions work on up to four heads, and two or four passes' loads
// in flight.  Lane l of a head holds elements 4 l .. 4 l + 3 of each half, so that
// where a whole head turns, both of a pair are the lane's own.
//   x' = x gamma / sqrt(mean(x^2) + eps);  (a, b) -> (a cos - b sin, b cos + a sin)
// The angle is pos * turns[i] mod 1, exact in 64-bit integers whatever the
// position, so only its last conversion to fp32 rounds.  Bound by the bytes of
// the rows for a prompt in fp32 (6 per element), by instruction issue in bf16
// (74 % of cycles, DRAM at 36 %), by the launch for a step.
// Measured, 4001 rows of 64 heads of 128: fp32 34.2 us (197 MB, 5.7 TB/s, 0.85
// of the measured copy), bf16 29.6 us (131 MB; 40 us with half the loads in
// flight).  A warp per head with four elements a lane issued three times the
// instructions and was bound by them (48 us).
template <typename SRC, typename DST, int D>
__global__ void __launch_bounds__(APPEND_THREADS, 7) qlin_append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int LANES = D / 8, PASS = APPEND_THREADS / LANES;  // lanes of a head, heads of a pass
  constexpr int AHEAD = sizeof(SRC) == 4 ? 2 : 4, H = D / 2;  // passes in flight: 64 bytes a thread
  __shared__ float2 cs[D / 2];                  // cos, sin of this row's angles
  __shared__ __align__(16) float gamma[2][D];   // of q, of k
  __shared__ float rows[PASS][D];
  const int row = blockIdx.x, b = row / p.step.T, t = row - b * p.step.T;
  const int at4 = threadIdx.x % LANES * 4, slot = threadIdx.x / LANES;  // this thread's elements, its head of a pass
  pdl_wait();
  pdl_launch_dependents();
  // everything that is read goes out before anything is waited for
  const int h1 = min((int)(blockIdx.y + 1) * p.heads_per_block, p.heads);
  const int h = blockIdx.y * p.heads_per_block + slot;
  // the heads of a token: of q, then of k, then of v
  const int v0 = p.Hq + p.cache.heads;
  const SRC* qs = static_cast<const SRC*>(p.q) + row * p.q_stride + at4;
  const SRC* ks = static_cast<const SRC*>(p.k) + (row * p.k_stride - (int64_t)p.Hq * D) + at4;
  const SRC* vs = static_cast<const SRC*>(p.v) + (row * p.v_stride - (int64_t)v0 * D) + at4;
  auto load = [&](Raw<SRC>& x, int head) { x.load((head < p.Hq ? qs : head < v0 ? ks : vs) + head * D, H); };
  Raw<SRC> x[AHEAD];
#pragma unroll
  for (int u = 0; u < AHEAD; u++)
    if (h + u * PASS < h1) load(x[u], h + u * PASS);
  const uint64_t turn = threadIdx.x < p.n_turns ? p.turns[threadIdx.x] : 0;
  for (int i = threadIdx.x; i < D; i += APPEND_THREADS) {
    gamma[0][i] = p.q_gamma ? p.q_gamma[i] : 1.f;
    gamma[1][i] = p.k_gamma ? p.k_gamma[i] : 1.f;
  }
  const int len = p.step.len[b], used = step_rows(p.step, b);
  const int depth = p.step.depth ? p.step.depth[b * p.step.tree_stride + t] : t;
  if (len < 0 || t >= used) return;
  const int n = p.n_turns;
  static_assert(APPEND_THREADS >= D / 2, "a thread per angle");
  if (threadIdx.x < n) {
    const int64_t angle = (int64_t)((uint64_t)((int64_t)len + depth) * turn);  // in [-1/2, 1/2) turns of 2^64
    float s, c;
    sincospif((float)(int32_t)(angle >> 32) * 0x1p-31f, &s, &c);
    cs[threadIdx.x] = make_float2(c, s);
  }
  const int64_t at = p.k ? token_offset(p.cache, p.step, b, (int64_t)len + t) : 0;
  if (at < 0 && threadIdx.x == 0) report(p.status, QLIN_ERR_BAD_INDEX);
  __syncthreads();
  // How a head turns: not at all; pairs, or whole halves, within the lane;
  // a power of two of whole lanes, with lane ^ flip; any other, through shared
  // memory.  The lane's cosines and sines are the same for all heads.
  const int flip = !p.pairs && n && n < H && n % 4 == 0 && (n & (n - 1)) == 0 && 2 * n <= H ? n / 4 : 0;
  const bool own = !p.pairs && n == H;
  float tc[4], ts[4];  // pairs: of elements 0 and 2 of each half; else of the first half's (flip: signed by its side)
#pragma unroll
  for (int e = 0; e < 4; e++) {
    int i = at4 + e;
    if (p.pairs) i = (e < 2 ? at4 + 2 * e : H + at4 + 2 * (e - 2)) / 2;
    const bool second = flip && i >= n;
    if (second) i -= n;
    const float2 w = i < n ? cs[i] : make_float2(1.f, 0.f);
    tc[e] = w.x;
    ts[e] = flip && !second ? -w.y : w.y;
  }
  DST* const qd = static_cast<DST*>(p.q_out) + row * p.q_out_stride + at4;
  auto finish = [&](float (&x)[8], int head) {
    const bool is_q = head < p.Hq, is_v = head >= v0, here = head < h1;
    if (__any_sync(0xFFFFFFFFu, here && !is_v)) {  // all lanes: the warp's heads may differ in kind
      if (p.q_gamma || p.k_gamma) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; e++) ss = fmaf(x[e], x[e], ss);
#pragma unroll
        for (int o = LANES / 2; o; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
        const float a = ss * (1.0f / D) + p.eps;
        float r = rsqrtf(a);  // and a Newton step, to one ulp (a = 0 or infinite: as it is)
        const float d = fmaf(-a * r, r, 1.f);
        if (fabsf(d) < 1.f) r = fmaf(0.5f * r, d, r);
        if ((is_q ? p.q_gamma : p.k_gamma) && !is_v) {
          const float* g = gamma[is_q ? 0 : 1] + at4;
          const float4 g0 = *reinterpret_cast<const float4*>(g), g1 = *reinterpret_cast<const float4*>(g + H);
          x[0] *= r * g0.x, x[1] *= r * g0.y, x[2] *= r * g0.z, x[3] *= r * g0.w;
          x[4] *= r * g1.x, x[5] *= r * g1.y, x[6] *= r * g1.z, x[7] *= r * g1.w;
        }
      }
      if (p.pairs) {
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const int i = e < 2 ? 2 * e : 4 + 2 * (e - 2);
          const float u = x[i], w = x[i + 1];
          if ((e < 2 ? at4 + 2 * e : H + at4 + 2 * (e - 2)) < 2 * n && !is_v) {
            x[i] = u * tc[e] - w * ts[e];
            x[i + 1] = w * tc[e] + u * ts[e];
          }
        }
      } else if (own) {
        if (!is_v)
#pragma unroll
          for (int e = 0; e < 4; e++) {
            const float u = x[e], w = x[4 + e];
            x[e] = u * tc[e] - w * ts[e];
            x[4 + e] = w * tc[e] + u * ts[e];
          }
      } else if (flip) {
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const float other = __shfl_xor_sync(0xFFFFFFFFu, x[e], flip);
          if (at4 < 2 * n && !is_v) x[e] = x[e] * tc[e] + other * ts[e];
        }
      } else if (n) {
        float* mine = rows[slot];
#pragma unroll
        for (int e = 0; e < 8; e++) mine[at4 + e % 4 + e / 4 * H] = x[e];
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 8; e++) {
          const int i = at4 + e % 4 + e / 4 * H;
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
      store4(x, qd + head * D);
      store4(x + 4, qd + head * D + H);
    } else if (at >= 0) {
      DST* dst = static_cast<DST*>(is_v ? p.cache.v : p.cache.k) + at + (head - (is_v ? v0 : p.Hq)) * p.cache.head_stride + at4;
      store4(x, dst);
      store4(x + 4, dst + H);
    }
  };
  const int warp_first = h - slot + (int)(threadIdx.x & ~31u) / LANES;  // the same in all lanes of a warp
  for (int off = 0; warp_first + off < h1; off += AHEAD * PASS) {
#pragma unroll
    for (int u = 0; u < AHEAD; u++) {
      const int head = h + off + u * PASS;
      if (warp_first + off + u * PASS >= h1) break;
      float now[8];
      x[u].get(now);
      if (head + AHEAD * PASS < h1) load(x[u], head + AHEAD * PASS);
      finish(now, head);
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
  if (q) {  // a row of q_out is written while other heads of q, k and v are still to be read
    const int64_t n = (int64_t)step->B * step->T, kv = cache->heads * D;
    const bool in_place = q_out == q && size == 2 && q_out_stride == q_stride;  // a thread writes what it alone read
    if ((!in_place && rows_overlap(q_out, q_out_stride * 2, Hq * D * 2, q, q_stride * size, Hq * D * size, n)) ||
        rows_overlap(q_out, q_out_stride * 2, Hq * D * 2, k, k_stride * size, kv * size, n) ||
        rows_overlap(q_out, q_out_stride * 2, Hq * D * 2, v, v_stride * size, kv * size, n))
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
  const int64_t pass = APPEND_THREADS / (D / 8);
  per = (per + pass - 1) / pass * pass;
  p.heads_per_block = (int)per;
  void* args[] = {&p};
  return launch_step(append_fn(src, cache->dtype, cache->width),
                     dim3((unsigned)rows, (unsigned)((p.heads + per - 1) / per), 1), dim3(APPEND_THREADS, 1, 1), 0,
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
