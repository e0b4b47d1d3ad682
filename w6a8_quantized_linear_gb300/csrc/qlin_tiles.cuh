// What the kernels that stream a paged cache through tensor cores share: the way
// from a CTA to its run of the items' tiles, TMA copies of pages, matrix
// descriptors and tensor memory.
#pragma once
#include <cuda.h>

#include "qlin_ptx.cuh"
#include "qlin_step.h"

namespace qlin {

__device__ __forceinline__ int64_t warp_sum64(int64_t v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// ---- runs ------------------------------------------------------------------------
//
// The (sequence, cache head) items' tiles of TILE tokens are laid end to end and
// cut into equal runs, one per CTA.  Work is measured in tiles, and GAP more
// between two items: what a CTA loses when its run goes on with another item.
// An item's n tiles are [start, start + n), and the gap follows.  P has the step,
// the cache, the number of CTAs, and tokens(b): what sequence b's items hold.

template <int TILE>
__device__ __forceinline__ int64_t tokens_to_tiles(int64_t n) { return (n + TILE - 1) / TILE; }
template <int TILE, int GAP, class P>
__device__ __forceinline__ int64_t work_of(const P& p, int64_t tiles) {  // a sequence's
  return tiles ? (tiles + GAP) * p.cache.heads : 0;
}
// Work of the sequences before b, and of all; a whole warp.
template <int TILE, int GAP, class P>
__device__ __forceinline__ void work_before(const P& p, int b, int64_t* before, int64_t* all) {
  const int lane = threadIdx.x & 31;
  int64_t x = 0, y = 0;
  for (int i = lane; i < p.step.B; i += 32) {
    const int64_t n = work_of<TILE, GAP>(p, tokens_to_tiles<TILE>(p.tokens(i)));
    y += n;
    if (i < b) x += n;
  }
  *before = warp_sum64(x);
  *all = warp_sum64(y);
}

// A CTA's run, item by item.
struct Walk {
  int64_t left;    // work of the run still ahead, this item's included
  int64_t tile;    // first tile of this item's part
  int64_t n;       // tiles of this part
  int64_t tokens;  // tokens of the sequence
  int b, h;
};
template <int TILE, int GAP, class P>
__device__ __forceinline__ void enter(const P& p, Walk& w) {  // the part of the item that w names
  const int64_t n = tokens_to_tiles<TILE>(w.tokens) - w.tile;
  w.n = n < w.left ? n : w.left;
}
template <int TILE, int GAP, class P>
__device__ __forceinline__ bool next_item(const P& p, Walk& w) {
  w.left -= w.n + GAP;
  if (w.left <= 0) return false;
  w.tile = 0;
  if (++w.h == p.cache.heads) {
    w.h = 0;
    do {
      if (++w.b >= p.step.B) return false;  // the run ends in the gap behind the last item
      w.tokens = p.tokens(w.b);
    } while (w.tokens == 0);
  }
  enter<TILE, GAP>(p, w);
  return true;
}
// Runs that work N is cut into: each at least one long, so that the CTAs
// between an item's first and last have all left a partial result of it.
template <class P>
__device__ __forceinline__ int runs_of(const P& p, int64_t N) { return N < p.ctas ? (int)N : p.ctas; }
// Where run c begins, floor(N c / runs), in 32 bits where they suffice.
__device__ __forceinline__ int64_t run_start(int64_t N, int c, int runs) {
  const int64_t x = N * c;
  return x >> 32 ? x / runs : (int64_t)((uint32_t)x / (uint32_t)runs);
}
// Where CTA c's run begins; a whole warp.  Up to 32 sequences' lengths are
// read once, in one trip.
template <int TILE, int GAP, class P>
__device__ __forceinline__ Walk first_item(const P& p, int c) {
  const int lane = threadIdx.x & 31;
  int64_t tokens = lane < p.step.B ? p.tokens(lane) : 0, all = work_of<TILE, GAP>(p, tokens_to_tiles<TILE>(tokens));
  for (int i = lane + 32; i < p.step.B; i += 32) all += work_of<TILE, GAP>(p, tokens_to_tiles<TILE>(p.tokens(i)));
  const int64_t N = warp_sum64(all);
  const int runs = runs_of(p, N);
  Walk w = {0, 0, 0, 0, 0, 0};
  if (c >= runs) return w;
  const int64_t x0 = run_start(N, c, runs);
  w.left = run_start(N, c + 1, runs) - x0;
  int64_t run = 0;
  for (int i0 = 0; i0 < p.step.B; i0 += 32) {
    if (i0) tokens = i0 + lane < p.step.B ? p.tokens(i0 + lane) : 0;
    const int64_t n = work_of<TILE, GAP>(p, tokens_to_tiles<TILE>(tokens));
    int64_t inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t a = __shfl_up_sync(0xFFFFFFFFu, inc, o);
      if (lane >= o) inc += a;
    }
    const uint32_t hit = __ballot_sync(0xFFFFFFFFu, x0 < run + inc);
    if (hit) {
      const int l = __ffs(hit) - 1;
      const int64_t start = __shfl_sync(0xFFFFFFFFu, run + inc - n, l);
      w.tokens = __shfl_sync(0xFFFFFFFFu, tokens, l);
      const int64_t tiles = tokens_to_tiles<TILE>(w.tokens), per = tiles + GAP;
      w.b = i0 + l;
      w.h = (int)run_start(x0 - start, 1, (int)per);  // tiles of one head: below 2^31
      w.tile = x0 - start - w.h * per;
      if (w.tile < tiles) {
        enter<TILE, GAP>(p, w);
      } else {  // in a gap: on with the item behind it
        w.left += w.tile - tiles;
        w.n = 0;
        if (!next_item<TILE, GAP>(p, w)) w.left = 0;
      }
      return w;
    }
    run += __shfl_sync(0xFFFFFFFFu, inc, 31);
  }
  w.left = 0;
  return w;
}
// The CTA whose run holds place x of N: floor(c N / runs) <= x < floor((c + 1) N / runs)
__device__ __forceinline__ int cta_of(int64_t x, int64_t N, int runs) {
  const int64_t y = (x + 1) * runs - 1;
  return (y | N) >> 32 ? (int)(y / N) : (int)((uint32_t)y / (uint32_t)N);
}

// ---- PTX -------------------------------------------------------------------------

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int token, int head, int page,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(dst),
      "l"(map), "r"(x), "r"(token), "r"(head), "r"(page), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::
          "r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// One lane of the warp, the same at every call.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}
// Matrix descriptor of a 128-byte-swizzled operand: rows of 64 16-bit values
// (128 bytes, on a 1024-byte boundary every eighth), `lbo` bytes between its
// 64-wide panels where the panels run along M or N, 1024 between groups of
// eight rows.
__device__ __forceinline__ uint64_t swizzled_desc(uint32_t addr, uint32_t lbo) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));  // below 2^-126: 0
  return y;
}

// ---- on the host -----------------------------------------------------------------

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder of tensor maps, or NULL.
inline EncodeTiled encode_tiled() {
  static const EncodeTiled fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) == cudaSuccess &&
        found == cudaDriverEntryPointSuccess)
      return reinterpret_cast<EncodeTiled>(f);
    (void)cudaGetLastError();
    return static_cast<EncodeTiled>(nullptr);
  }();
  return fn;
}

// [pages, heads, page_size, width] as boxes of 64 elements x `box` tokens,
// 128-byte swizzled
inline bool encode(EncodeTiled encode_tiled, CUtensorMap* map, const qlin_kv_cache* c, void* base, int box) {
  const cuuint64_t dims[4] = {(cuuint64_t)c->width, (cuuint64_t)c->page_size, (cuuint64_t)c->heads,
                              (cuuint64_t)c->pages};
  const cuuint64_t strides[3] = {(cuuint64_t)c->token_stride * 2, (cuuint64_t)c->head_stride * 2,
                                 (cuuint64_t)c->page_stride * 2};
  const cuuint32_t shape[4] = {64, (cuuint32_t)box, 1, 1}, one[4] = {1, 1, 1, 1};
  return encode_tiled(map, c->dtype == QLIN_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                  base, dims, strides, shape, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace qlin
