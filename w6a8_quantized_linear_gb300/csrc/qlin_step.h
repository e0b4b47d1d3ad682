// What the kernels of a decode step share: the cache and the step as kernel
// parameters, the way from a token to its place in the cache, conversions to
// and from the cache's types, and the host-side checks of both structs.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "qlin.h"

namespace qlin {

constexpr int64_t STEP_WS_HEADER = 256;  // the status word and reserved bytes

inline bool is_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline qlin_status status_of(cudaError_t e) {
  if (e == cudaSuccess) return QLIN_OK;
  (void)cudaGetLastError();
  return QLIN_ERR_CUDA;
}

inline qlin_status check_cache(const qlin_kv_cache* c) {
  if (!c) return QLIN_ERR_INVALID_ARG;
  if (c->dtype != QLIN_BF16 && c->dtype != QLIN_F16) return QLIN_ERR_INVALID_ARG;
  if (c->heads < 1 || c->pages < 1 || c->pages > 0x7FFFFFFF) return QLIN_ERR_INVALID_ARG;
  if (!c->k || !c->v || !is_aligned(c->k, 16) || !is_aligned(c->v, 16)) return QLIN_ERR_INVALID_ARG;
  if (c->width != 64 && c->width != 128 && c->width != 256) return QLIN_ERR_UNSUPPORTED;
  if (c->heads > 1024) return QLIN_ERR_UNSUPPORTED;
  if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1))) return QLIN_ERR_UNSUPPORTED;
  const int64_t strides[3] = {c->page_stride, c->head_stride, c->token_stride};
  for (int64_t s : strides)
    if (s < 1 || s % 8 || s > (int64_t(1) << 36)) return QLIN_ERR_INVALID_ARG;
  if (c->token_stride < c->width) return QLIN_ERR_INVALID_ARG;
  return QLIN_OK;
}

// max_t: the most rows per sequence that the call takes
inline qlin_status check_step(const qlin_kv_step* s, int64_t max_t) {
  if (!s || s->B < 0 || s->T < 0) return QLIN_ERR_INVALID_ARG;
  if (s->B == 0 || s->T == 0) return QLIN_OK;  // an empty step: nothing is read
  if (!s->page_table || !is_aligned(s->page_table, 4) || !s->len || !is_aligned(s->len, 4)) return QLIN_ERR_INVALID_ARG;
  if (s->max_pages < 1 || s->table_stride < s->max_pages) return QLIN_ERR_INVALID_ARG;
  if (!is_aligned(s->count, 4) || !is_aligned(s->depth, 4) || !is_aligned(s->mask, 4)) return QLIN_ERR_INVALID_ARG;
  if (s->tree_stride < 0 || (s->tree_stride != 0 && s->tree_stride < s->T)) return QLIN_ERR_INVALID_ARG;
  if (s->T > max_t || (int64_t)s->B * s->T > 0x7FFFFFFF) return QLIN_ERR_UNSUPPORTED;
  return QLIN_OK;
}

// rows of `width` elements of `size` bytes, `stride` elements apart, each on a
// 16-byte boundary
inline bool rows_ok(const void* p, int64_t stride, int64_t width, int64_t size) {
  return p && is_aligned(p, 16) && stride >= width && (stride * size) % 16 == 0;
}

// Whether n rows of wa bytes, sa bytes apart from a on, share a byte with n rows
// of wb bytes, sb apart from b on (rows of unequal strides: the ranges they lie
// in).  wa <= sa, wb <= sb.
inline bool rows_overlap(const void* a, int64_t sa, int64_t wa, const void* b, int64_t sb, int64_t wb, int64_t n) {
  using wide = __int128;
  if (!a || !b || n < 1) return false;
  const wide ahead = (wide)reinterpret_cast<uintptr_t>(b) - (wide)reinterpret_cast<uintptr_t>(a);
  if (ahead >= (wide)(n - 1) * sa + wa || -ahead >= (wide)(n - 1) * sb + wb) return false;
  if (n == 1 || sa != sb) return true;
  // the first k > -n for which row i + k of b does not end before row i of a begins
  const wide gap = -ahead - wb;
  wide k = gap / sa - (gap % sa < 0) + 1;
  if (k < 1 - n) k = 1 - n;
  return k < n && ahead + k * sa < wa;
}

// Accumulated scores: [B, heads, room] 32-bit values, the strides in elements; no
// two items share a place.
inline bool scores_ok(int64_t B, int64_t heads, int64_t room, int64_t seq_stride, int64_t head_stride) {
  if (seq_stride < 0 || head_stride < 0 || seq_stride > (int64_t(1) << 40) || head_stride > (int64_t(1) << 40)) return false;
  const bool heads_inside = head_stride >= room && (B == 1 || seq_stride >= (heads - 1) * head_stride + room);
  const bool seqs_inside = seq_stride >= room && (heads == 1 || head_stride >= (B - 1) * seq_stride + room);
  return (heads == 1 || head_stride >= room) && (B == 1 || seq_stride >= room) &&
         (heads == 1 || B == 1 || heads_inside || seqs_inside);
}
inline int64_t scores_span(int64_t B, int64_t heads, int64_t room, int64_t seq_stride, int64_t head_stride) {
  return (B - 1) * seq_stride + (heads - 1) * head_stride + room;
}

inline qlin_status check_status_ws(const void* ws, size_t ws_bytes) {  // an optional workspace
  if (!ws) return QLIN_OK;
  if (!is_aligned(ws, 256)) return QLIN_ERR_INVALID_ARG;
  return ws_bytes < (size_t)STEP_WS_HEADER ? QLIN_ERR_WORKSPACE : QLIN_OK;
}

inline qlin_status launch_step(const void* fn, dim3 grid, dim3 block, size_t smem, cudaStream_t s, void** args,
                               bool pdl, int cluster_x = 1) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (cluster_x > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = (unsigned)cluster_x;
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    n++;
  }
  if (pdl) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    n++;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return status_of(cudaLaunchKernelExC(&cfg, fn, args));
}

// ---- on the device ------------------------------------------------------------

__device__ __forceinline__ int step_rows(const qlin_kv_step& s, int b) {  // rows in use
  if (!s.count) return s.T;
  const int n = s.count[b];
  return n < 0 ? 0 : n > s.T ? s.T : n;
}
__device__ __forceinline__ uint32_t step_mask(const qlin_kv_step& s, int b, int t) {
  if (!s.mask) return 0xFFFFFFFFu >> (31 - t);
  return (uint32_t)s.mask[b * s.tree_stride + t];
}
// Element offset of a token's row in k and v, without its head; -1 where the
// page is out of range.
__device__ __forceinline__ int64_t token_offset(const qlin_kv_cache& c, const qlin_kv_step& s, int b, int64_t token) {
  const int shift = 31 - __clz(c.page_size);  // a power of two
  const int64_t slot = token >> shift;
  if (slot >= s.max_pages) return -1;
  const int page = s.page_table[b * s.table_stride + slot];
  if (page < 0 || page >= c.pages) return -1;
  return page * c.page_stride + (token & (c.page_size - 1)) * c.token_stride;
}
__device__ __forceinline__ void report(uint32_t* status, uint32_t what) {
  if (status) atomicCAS(status, 0u, what);  // the first finding stays
}

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
  const __half2 r = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ float2 unpack2(uint32_t w, __nv_bfloat16) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ float2 unpack2(uint32_t w, __half) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

}  // namespace qlin
