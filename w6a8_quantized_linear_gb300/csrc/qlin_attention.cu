// qlin_tree_attention: a step's rows over the paged cache.
#include <cmath>

#include "qlin_ptx.cuh"
#include "qlin_step.h"

namespace qlin {
namespace {

constexpr int ATT_WARPS = 4;

struct AttentionParams {
  qlin_kv_cache cache;
  qlin_kv_step step;
  const void* q;
  void* out;
  int64_t q_stride, out_stride;
  uint32_t* status;
  float scale_log2;  // scale * log2(e): weights are powers of two
  int Hq;
};

// One block per row and query head, each warp every fourth token, with the
// running maximum and sum; the warps' partial results joined at the end.
template <typename T, int D>
__global__ void __launch_bounds__(ATT_WARPS * 32) qlin_attention_kernel(const __grid_constant__ AttentionParams p) {
  __shared__ float part[ATT_WARPS][D + 2];
  constexpr int E = D / 32;
  const int row = blockIdx.x, head = blockIdx.y;
  const int b = row / p.step.T, t = row - b * p.step.T;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_launch_dependents();
  const int len = p.step.len[b];
  const int rows = step_rows(p.step, b);
  if (len < 0 || t >= rows) return;
  const uint32_t mask = step_mask(p.step, b, t);
  const int hk = head / (p.Hq / p.cache.heads);
  float q[E], o[E], m = -INFINITY, l = 0.f;
  const T* qp = static_cast<const T*>(p.q) + row * p.q_stride + (int64_t)head * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    const float2 f = unpack2(*reinterpret_cast<const uint32_t*>(qp + e), T());
    q[e] = f.x * p.scale_log2, q[e + 1] = f.y * p.scale_log2;
    o[e] = o[e + 1] = 0.f;
  }
  for (int64_t j = warp; j < (int64_t)len + rows; j += ATT_WARPS) {
    if (j >= len && !(mask >> (j - len) & 1)) continue;
    const int64_t at = token_offset(p.cache, p.step, b, j);
    if (at < 0) {
      if (lane == 0) report(p.status, QLIN_ERR_BAD_INDEX);
      continue;
    }
    const T* kp = static_cast<const T*>(p.cache.k) + at + hk * p.cache.head_stride + lane * E;
    const T* vp = static_cast<const T*>(p.cache.v) + at + hk * p.cache.head_stride + lane * E;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const float2 f = unpack2(*reinterpret_cast<const uint32_t*>(kp + e), T());
      s = fmaf(q[e], f.x, fmaf(q[e + 1], f.y, s));
    }
#pragma unroll
    for (int i = 16; i; i >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, i);
    const float mn = fmaxf(m, s);
    const float keep = m == mn ? 1.f : exp2f(m - mn), w = exp2f(s - mn);
    m = mn;
    l = l * keep + w;
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const float2 f = unpack2(*reinterpret_cast<const uint32_t*>(vp + e), T());
      o[e] = fmaf(w, f.x, o[e] * keep), o[e + 1] = fmaf(w, f.y, o[e + 1] * keep);
    }
  }
#pragma unroll
  for (int e = 0; e < E; e++) part[warp][lane * E + e] = o[e];
  if (lane == 0) part[warp][D] = m, part[warp][D + 1] = l;
  __syncthreads();
  float mx = -INFINITY, sum = 0.f;
  for (int w = 0; w < ATT_WARPS; w++) mx = fmaxf(mx, part[w][D]);
  float f[ATT_WARPS];
  for (int w = 0; w < ATT_WARPS; w++) {
    f[w] = part[w][D] == -INFINITY ? 0.f : exp2f(part[w][D] - mx);
    sum += f[w] * part[w][D + 1];
  }
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + row * p.out_stride + (int64_t)head * D;
  for (int e = threadIdx.x; e < D; e += ATT_WARPS * 32) {
    float x = 0.f;
    for (int w = 0; w < ATT_WARPS; w++)
      if (f[w] != 0.f) x += f[w] * part[w][e];
    out[e] = __float2bfloat16(sum == 0.f ? 0.f : x / sum);
  }
}

const void* attention_fn(int dtype, int width) {
  if (dtype == QLIN_BF16)
    return width == 64    ? reinterpret_cast<const void*>(qlin_attention_kernel<__nv_bfloat16, 64>)
           : width == 128 ? reinterpret_cast<const void*>(qlin_attention_kernel<__nv_bfloat16, 128>)
                          : reinterpret_cast<const void*>(qlin_attention_kernel<__nv_bfloat16, 256>);
  return width == 64    ? reinterpret_cast<const void*>(qlin_attention_kernel<__half, 64>)
         : width == 128 ? reinterpret_cast<const void*>(qlin_attention_kernel<__half, 128>)
                        : reinterpret_cast<const void*>(qlin_attention_kernel<__half, 256>);
}

qlin_status check_heads(const qlin_kv_cache* c, int64_t B, int64_t T, int Hq) {
  if (B < 0 || T < 0 || Hq < 1 || Hq % c->heads) return QLIN_ERR_INVALID_ARG;
  if (T > QLIN_MAX_TREE || T * (Hq / c->heads) > 128) return QLIN_ERR_UNSUPPORTED;
  return QLIN_OK;
}

}  // namespace
}  // namespace qlin

using namespace qlin;

extern "C" {

qlin_status qlin_tree_attention_workspace_bytes(const qlin_kv_cache* cache, int B, int T, int Hq, size_t* bytes) {
  qlin_status st = check_cache(cache);
  if (st != QLIN_OK) return st;
  st = check_heads(cache, B, T, Hq);
  if (st != QLIN_OK) return st;
  if (!bytes) return QLIN_ERR_INVALID_ARG;
  *bytes = (size_t)STEP_WS_HEADER;
  return QLIN_OK;
}

qlin_status qlin_tree_attention(const qlin_kv_cache* cache, const qlin_kv_step* step, int Hq, const void* q,
                                int64_t q_stride, float scale, void* out, int64_t out_stride, void* ws,
                                size_t ws_bytes, unsigned flags, void* stream) {
  qlin_status st = check_cache(cache);
  if (st != QLIN_OK) return st;
  st = check_step(step, QLIN_MAX_TREE);
  if (st != QLIN_OK) return st;
  size_t need = 0;
  st = qlin_tree_attention_workspace_bytes(cache, step->B, step->T, Hq, &need);
  if (st != QLIN_OK) return st;
  if (flags & ~QLIN_FLAG_PDL) return QLIN_ERR_INVALID_ARG;
  if (!std::isfinite(scale)) return QLIN_ERR_INVALID_ARG;
  if (step->B == 0 || step->T == 0) return QLIN_OK;
  const int64_t D = cache->width;
  if (!rows_ok(q, q_stride, Hq * D, 2) || !rows_ok(out, out_stride, Hq * D, 2)) return QLIN_ERR_INVALID_ARG;
  if (!ws || !is_aligned(ws, 256)) return QLIN_ERR_INVALID_ARG;
  if (ws_bytes < need) return QLIN_ERR_WORKSPACE;
  AttentionParams p = {*cache, *step,      q, out, q_stride, out_stride, static_cast<uint32_t*>(ws),
                       scale * 1.4426950408889634f, Hq};
  void* args[] = {&p};
  return launch_step(attention_fn(cache->dtype, cache->width), dim3((unsigned)(step->B * step->T), (unsigned)Hq, 1),
                     dim3(ATT_WARPS * 32, 1, 1), 0, static_cast<cudaStream_t>(stream), args,
                     (flags & QLIN_FLAG_PDL) != 0);
}

}  // extern "C"
