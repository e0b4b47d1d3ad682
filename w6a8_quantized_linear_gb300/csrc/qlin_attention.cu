// qlin_tree_attention: a step's rows over the paged cache.
//
// Two launches.  The first streams the committed tokens: their (sequence,
// cache head) items' tiles are laid end to end and cut into equal runs, one
// per CTA, whatever the lengths are, and each CTA leaves unnormalised partial
// results of the items it touched.  Every row sees all of these tokens, so no
// mask enters.  The second joins an item's partial results with the step's own
// rows (at most 32 keys, under the tree's mask, on the CUDA cores, each row
// reading only the keys that it sees) and normalises; it computes the scores
// of those while the first still runs.
#include <cmath>
#include <mutex>
#include <type_traits>
#include <utility>

#include "qlin_tiles.cuh"

namespace qlin {
namespace {

constexpr int ATT_THREADS = 224;   // four softmax warps, then the producer, MMA and cleaner warps
constexpr int PRODUCER = 4, ISSUER = 5, CLEANER = 6;
constexpr int ATT_ROWS = 128;      // query rows of an item at most: the lanes of tensor memory
constexpr int ATT_MAX_CTAS = 160;  // the workspace holds the partial results of this many (one per SM)
constexpr int JOIN_THREADS = 512;
constexpr float RESCALE_AT = 8.f;  // log2 units that a row's maximum may rise before its sums are rescaled
// Weights are relative to a reference that lies so many log2 units below the
// maximum that set it: fp16 holds 2^(7 + RESCALE_AT), and its smallest steps
// are then 2^-31 of the largest weight instead of 2^-24.  (200000 tokens of
// 2^-25.6 each were all rounded away from the sums of v, and counted in l.)
template <typename T>
constexpr float BELOW = std::is_same<T, __half>::value ? 7.f : 0.f;
// From here on fp32 scores (log2 units) are a step or more apart.
constexpr float FAR = 0x1p23f;

// Tokens of a tile: 32 KB of keys and of values (16 KB at width 64).
__host__ __device__ constexpr int tile_tokens(int width) { return width == 256 ? 64 : 128; }
__host__ __device__ constexpr int tile_bytes(int width) { return tile_tokens(width) * width * 2; }
__host__ __device__ constexpr int q_bytes(int width) { return ATT_ROWS * width * 2; }
// Ring buffers beside the query rows: 200 KB together, so that blocks of the
// second launch find room on the SM (threads and registers likewise) and form
// their scores while the first still runs.
__host__ __device__ constexpr int ring_buffers(int width) { return (200 * 1024 - q_bytes(width)) / tile_bytes(width); }
constexpr int MAX_RING = 11;

struct AttentionParams {
  CUtensorMap map_k, map_v, map_q;
  qlin_kv_cache cache;
  qlin_kv_step step;
  const void* q;
  __nv_bfloat16* out;
  int64_t q_stride, out_stride;
  uint32_t* status;
  float* partial;    // [slot][width + 2][padded rows]: sums, then references (log2 units) and weights' sums
  float scale_log2;  // scale * log2(e): weights are powers of two
  int group, R, Rp;  // query heads of a cache head; query rows of an item: T * group, padded to 8
  int ctas;
  int box;           // tokens per TMA copy: a page or a tile, whichever is smaller
  int page_shift;    // log2 of the page size
  int64_t fault_copy;  // test only (FAULT): the copy that the first CTA never issues
  float* stats;      // the rows' references and sums of weights, or none

  __device__ __forceinline__ int64_t tokens(int b) const {  // the committed ones that are there
    const int64_t len = step.len[b];
    if (len <= 0 || step_rows(step, b) == 0) return 0;
    const int64_t most = (int64_t)step.max_pages * cache.page_size;
    return len < most ? len : most;
  }
};

// Work of a change to another item: 5 to 7 us (the sums' way out of tensor memory,
// other query rows, the pipeline filled again) against 1.5 us for a tile; with 1,
// 2, 3, 4 and 6, five items of 275 tiles took 31.1, 29.9, 28.9, 29.5 and 29.2 us,
// 152 of 4 to 14 tiles 33.5, 32.0, 30.8, 31.5 and 32.2.
constexpr int GAP = 3;

// A barrier of the four softmax warps that tells all of them whether all are
// still at work (every wait before it is bounded, so all four reach it).
__device__ __forceinline__ bool softmax_bar(bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.and.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"((uint32_t)ok)
      : "memory");
  return all != 0;
}

__device__ __forceinline__ void softmax_sync() { asm volatile("barrier.cta.sync 1, 128;" ::: "memory"); }

struct AttentionShared {
  uint64_t full[MAX_RING], empty[MAX_RING];
  uint64_t s_full[2], s_free[2], p_full[2], p_free[2];
  uint64_t q_full, o_full, v_dirty, v_clean, drained;
  uint32_t tmem;
  int dead;  // a wait has expired: every role leaves its loop
  Walk walk;
  float m[ATT_ROWS], l[ATT_ROWS];  // each lane's reference and sum of weights at an item's end
};

// A bounded wait of one role; on expiry the workspace's status word is set and
// all roles leave.
__device__ __forceinline__ bool role_wait(uint64_t* bar, uint32_t parity, AttentionShared* s, uint32_t* status) {
  if (mbar_try_wait(bar, parity)) return true;
  if (!*(volatile int*)&s->dead && mbar_wait(bar, parity)) return true;
  s->dead = 1;
  report(status, QLIN_ERR_DEVICE_TIMEOUT);
  return false;
}

// The committed tokens.  S = Q K^T (128 query lanes x a tile's tokens) and
// O += P V on tcgen05 with fp32 accumulators in tensor memory: lane = query
// row, so that a softmax thread owns a row and needs no exchange.  P goes from
// registers into tensor memory in the cache's type (half a step each, 2^-8 of a
// weight in bf16: both operands of a product have one type, and weights in two
// parts would need tensor memory that scores and sums take, and half as many
// products again; their sum l adds them unrounded in fp32) and is the A operand
// of the second product; keys and values are read by the tensor cores straight
// from the ring that TMA fills (128-byte swizzle; V as the transposed operand).
//
// Bound by the stream of keys and values: a tile's 64 KB take an SM 1.5 us at
// the measured copy bandwidth, its products 0.5 to 0.7 us, its softmax 0.6 us
// where the warps share it.  Measured (both launches): 48 query rows over
// 131k tokens of 4 heads of 256, 95.8 us for 537 MB (5.6 TB/s, 0.82 of the
// copy; the stream itself runs at 0.97, the rest is start, joining and the
// SMs' different ends); 18 rows over 8 sequences of 8 heads of 128, 111 us for
// 661 MB (0.88); width 64 streams 0.62 to 0.66 of the copy, bound by the
// softmax's latency per tile.
//
// A warp reaches 32 lanes, so with few rows most softmax warps would idle while
// one takes longer over a tile (128 tokens: 1.9 us when this was measured) than
// the tile's bytes take.  SPLIT = 2 or 4 therefore lays the query
// rows down that many times (up to 64 or 32 rows), and each copy's warps take
// their own part of a tile's tokens: P is zero elsewhere, once and for all, and
// each copy's lanes of O hold its tokens' sums, which are added at the item's
// end.
//
// A row's maximum may grow by 2^8 before its sums are rescaled in tensor
// memory: weights are relative to a maximum of the past (in fp16 to 2^-7 of
// it), at most 2^8 (2^15), which fp16 holds.
// (At most 128 registers, so that blocks of the second launch find room beside.)
template <typename T, int D, int SPLIT, bool FAULT = false>
__global__ void __launch_bounds__(ATT_THREADS, 2) qlin_attention_kernel(const __grid_constant__ AttentionParams p) {
  extern __shared__ uint8_t raw[];
  __shared__ AttentionShared sh;
  constexpr int TK = tile_tokens(D), TB = tile_bytes(D), NB = ring_buffers(D), PANELS = D / 64;
  constexpr uint32_t O_COL = 0, S_COL = D, P_COL = D + 2 * TK;  // columns of tensor memory
  static_assert(P_COL + TK <= 512 && NB >= 4 && NB <= MAX_RING, "tensor memory and ring");
  AttentionShared* s = &sh;
  const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
  const uint32_t q_smem = base, ring = base + q_bytes(D);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int LANES = ATT_ROWS / SPLIT, CW = TK / SPLIT;  // rows of a copy, tokens of a tile that it takes
  const int active = SPLIT > 1 ? 4 : (p.R + 31) / 32;      // softmax warps with rows

  if (threadIdx.x == 0) {
    for (int i = 0; i < NB; i++) mbar_init(&s->full[i], 1), mbar_init(&s->empty[i], 1);
    for (int i = 0; i < 2; i++) {
      mbar_init(&s->s_full[i], 1);
      mbar_init(&s->s_free[i], active);
      mbar_init(&s->p_full[i], active);
      mbar_init(&s->p_free[i], 1);
    }
    mbar_init(&s->q_full, 1);
    mbar_init(&s->o_full, 1);
    mbar_init(&s->v_dirty, 1);
    mbar_init(&s->v_clean, 1);
    mbar_init(&s->drained, 1);
    s->dead = 0;
    mbar_fence_init();
  }
  if (warp == ISSUER) tmem_alloc(&s->tmem, 512);
  pdl_wait();
  pdl_launch_dependents();
  if (warp == PRODUCER) {
    const Walk w = first_item<TK, GAP>(p, blockIdx.x);
    if (lane == 0) s->walk = w;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s->tmem;
  Walk w = s->walk;

  if (w.left > 0) {
    if (warp == PRODUCER) {
      // ---- producer: a lane per TMA copy (a page's or a tile's rows of one 64-wide panel)
      constexpr uint32_t row_bytes = 128;
      const int boxes = TK / p.box, copies = boxes * PANELS;  // <= 16
      const int box = lane % boxes, panel = lane / boxes;
      uint32_t i = 0;  // ring position
      bool ok = true;
      do {
        // page indexes are read a tile ahead
        const int32_t* table = p.step.page_table + w.b * p.step.table_stride;
        int64_t token = w.tile * TK + box * p.box;
        int next = lane < copies && token < w.tokens ? table[token >> p.page_shift] : -1;
        for (int64_t t = 0; t < w.n && ok; t++, token += TK) {
          int page = next;
          if (lane < copies && token < w.tokens && (page < 0 || page >= p.cache.pages)) {
            page = -1;
            report(p.status, QLIN_ERR_BAD_INDEX);
          }
          next = t + 1 < w.n && lane < copies && token + TK < w.tokens ? table[(token + TK) >> p.page_shift] : -1;
          const uint32_t bytes = __popc(__ballot_sync(0xFFFFFFFFu, page >= 0)) * p.box * row_bytes;
          for (int kv = 0; kv < 2; kv++, i++) {
            const uint32_t slot = i % NB, use = i / NB;
            if (use) ok = role_wait(&s->empty[slot], (use - 1) & 1, s, p.status);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(&s->full[slot], bytes);
            __syncwarp();
            const bool lost = FAULT && blockIdx.x == 0 && i == p.fault_copy;  // test only: this phase never completes
            if (page >= 0 && !lost)
              tma_load_4d(ring + slot * TB + (panel * TK + box * p.box) * 128, kv ? &p.map_v : &p.map_k, panel * 64,
                          (int)(token & (p.cache.page_size - 1)), w.h, page, &s->full[slot]);
          }
        }
      } while (ok && next_item<TK, GAP>(p, w));
      // nothing leaves while its copies are in flight, whichever role gave up
      // (this one may have issued its last copy long before); where none did,
      // they are all waited for elsewhere too
      for (uint32_t j = i > NB ? i - NB : 0; j < i; j++) (void)mbar_wait(&s->full[j % NB], (j / NB) & 1);
    } else if (warp == ISSUER) {
      // ---- MMA: the whole warp keeps the books, so that descriptors stay in
      // uniform registers, and one elected thread issues (built by that thread
      // alone they cost it 70 cycles an MMA, and it bound the kernel)
      constexpr uint32_t type = std::is_same<T, __nv_bfloat16>::value ? (1u << 7) | (1u << 10) : 0u;
      constexpr uint32_t id_s = mma_idesc_f16(128, TK) | type;
      constexpr uint32_t id_o = mma_idesc_f16(128, D) | type | (1u << 16);  // B along N
      uint32_t n = 0, seg = 0, dirty = 0;
      uint32_t ks = 0, kp = 0, vs = 1, vp = 0;  // ring places of the next keys and values, and their parities
      bool ok = true;
      do {
        ok = __all_sync(0xFFFFFFFFu, role_wait(&s->q_full, seg & 1, s, p.status));
        const int tiles = __shfl_sync(0xFFFFFFFFu, (int)w.n, 0);
        const int full_tiles = __shfl_sync(0xFFFFFFFFu, (int)min(w.n, w.tokens / TK - w.tile), 0);
        tc_fence_after();
        for (int t = 0; t <= tiles && ok; t++) {
          if (t < tiles) {  // S(t)
            const uint32_t m = __shfl_sync(0xFFFFFFFFu, n + t, 0);
            ok = role_wait(&s->full[ks], kp, s, p.status);
            if (ok && m >= 2) ok = role_wait(&s->s_free[m & 1], ((m >> 1) - 1) & 1, s, p.status);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            tc_fence_after();
            const uint32_t slot = __shfl_sync(0xFFFFFFFFu, ks, 0), kb = ring + slot * TB;
            if (elect_one()) {
#pragma unroll
              for (int e = 0; e < D / 16; e++)
                mma_smem_a(tmem + S_COL + (m & 1) * TK,
                           swizzled_desc(q_smem + (e / 4) * (ATT_ROWS * 128) + (e % 4) * 32, 16),
                           swizzled_desc(kb + (e / 4) * (TK * 128) + (e % 4) * 32, 16), id_s, e > 0);
              mma_commit(&s->empty[slot]);
              mma_commit(&s->s_full[m & 1]);
            }
            __syncwarp();
            ks += 2;
            if (ks >= NB) ks -= NB, kp ^= 1;
          }
          if (t > 0) {  // O += P(t - 1) V(t - 1)
            const uint32_t m = __shfl_sync(0xFFFFFFFFu, n + t - 1, 0);
            ok = role_wait(&s->full[vs], vp, s, p.status);
            const bool ragged = t > full_tiles;  // the sequence's last tile, not full
            if (ok && ragged && lane == 0) mbar_arrive(&s->v_dirty);
            if (ok) ok = role_wait(&s->p_full[m & 1], (m >> 1) & 1, s, p.status);
            if (ok && ragged) ok = role_wait(&s->v_clean, dirty++ & 1, s, p.status);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            tc_fence_after();
            const uint32_t slot = __shfl_sync(0xFFFFFFFFu, vs, 0), vb = ring + slot * TB;
            if (elect_one()) {
#pragma unroll
              for (int e = 0; e < TK / 16; e++)
                mma_tmem_a(tmem + O_COL, tmem + P_COL + (m & 1) * (TK / 2) + e * 8, swizzled_desc(vb + e * 2048, TK * 128),
                           id_o, t > 1 || e > 0);
              mma_commit(&s->empty[slot]);
              mma_commit(&s->p_free[m & 1]);
              if (t == tiles) mma_commit(&s->o_full);
            }
            __syncwarp();
            vs += 2;
            if (vs >= NB) vs -= NB, vp ^= 1;
          }
        }
        n += tiles;
        seg++;
      } while (ok && next_item<TK, GAP>(p, w));
      if (!ok && elect_one()) {  // the products in flight end before tensor memory is freed
        mma_commit(&s->drained);
        (void)mbar_wait(&s->drained, 0);
      }
    } else if (warp == CLEANER) {
      // ---- cleaner: the rows behind the last token hold whatever the page or
      // the ring held; their weight is 0, but 0 * NaN is not.  Asked for each
      // ragged tile once its copies have landed.
      uint32_t n = 0, dirty = 0;
      bool ok = true;
      do {
        n += (uint32_t)w.n;
        const int64_t end = (w.tile + w.n) * TK;
        if (end > w.tokens) {
          ok = __all_sync(0xFFFFFFFFu, role_wait(&s->v_dirty, dirty++ & 1, s, p.status));
          if (!ok) break;
          const uint32_t v = ring + ((2 * n - 1) % NB) * TB;
          const int valid = (int)(w.tokens - (end - TK)), units = (TK - valid) * 8;
          for (int c = lane; c < PANELS * units; c += 32)
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(v + ((c / units) * TK + valid) * 128 +
                                                                          (c % units) * 16),
                         "r"(0)
                         : "memory");
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s->v_clean);
        }
      } while (next_item<TK, GAP>(p, w));
    } else {
      // ---- softmax: a thread per query row
      const int at = threadIdx.x, row = at % LANES, copy = at / LANES;  // `at`: the lane of tensor memory
      const bool live = row < p.R;
      const uint32_t lanes = (uint32_t)(warp * 32) << 16;
      uint32_t n = 0, seg = 0;
      bool ok = true;
      if (SPLIT > 1) {  // the other copies' tokens
        uint32_t zero[32];
#pragma unroll
        for (int e = 0; e < 32; e++) zero[e] = 0;
#pragma unroll
        for (int c = 0; c < TK; c += 32) tmem_st32(tmem + lanes + P_COL + c, zero);
        tmem_wait_st();
      }
      do {
        if (at == 0) {  // the item's query rows, T x group of them, once per copy
          mbar_arrive_expect_tx(&s->q_full, (uint32_t)(SPLIT * PANELS * p.R * 128));
#pragma unroll
          for (int k = 0; k < SPLIT; k++)
#pragma unroll
            for (int e = 0; e < PANELS; e++)
              tma_load_3d(q_smem + e * (ATT_ROWS * 128) + k * LANES * 128, &p.map_q, e * 64, w.h * p.group, w.b * p.step.T,
                          &s->q_full);
        }
        float m_used = -INFINITY, l = 0.f;  // the reference, the sum of weights relative to it
        if (warp < active) {
          for (int64_t t = 0; t < w.n; t++) {
            const uint32_t m = n + (uint32_t)t;
            ok = __all_sync(0xFFFFFFFFu, role_wait(&s->s_full[m & 1], (m >> 1) & 1, s, p.status));
            if (!ok) break;
            tc_fence_after();
            // 32 scores at a time: the maximum first, then (read again, but for
            // the last 32) the weights
            constexpr int CX = CW < 32 ? CW : 32;
            const int64_t ahead = w.tokens - (w.tile + t) * TK - copy * CW;  // of this copy's tokens, those that are there
            const int valid = ahead < CW ? (int)ahead : CW;
            const uint32_t st = tmem + lanes + S_COL + (m & 1) * TK + copy * CW;
            float x[CX];
            auto scores = [&](int c0) {
              if constexpr (CX < 32)
                tmem_ld16(st + c0, *reinterpret_cast<uint32_t(*)[16]>(x));
              else
                tmem_ld32(st + c0, reinterpret_cast<uint32_t*>(x));
              tmem_wait_ld();
            };
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c0 = 0; c0 < CW; c0 += CX) {
              scores(c0);
              if (valid < CW) {
#pragma unroll
                for (int c = 0; c < CX; c++)
                  if (c0 + c < valid) mx[c & 3] = fmaxf(mx[c & 3], x[c] * p.scale_log2);
              } else {
#pragma unroll
                for (int c = 0; c < CX; c++) mx[c & 3] = fmaxf(mx[c & 3], x[c] * p.scale_log2);
              }
            }
            const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            float keep = 1.f;
            bool rescale = false;
            const float ref = fabsf(mt) < FAR ? mt - BELOW<T> : mt;
            if (t == 0) {
              m_used = ref;
            } else if (ref > m_used + RESCALE_AT) {
              keep = exp2_approx(m_used - ref);
              m_used = ref;
              l *= keep;
              rescale = live;
            }
            // the sums in tensor memory, where a row's maximum rose: once the
            // product before this one has been added
            if (__any_sync(0xFFFFFFFFu, rescale)) {
              ok = __all_sync(0xFFFFFFFFu, role_wait(&s->p_free[(m - 1) & 1], ((m - 1) >> 1) & 1, s, p.status));
              if (!ok) break;
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                tmem_ld32(tmem + lanes + O_COL + c, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; e++) o[e] = __float_as_uint(__uint_as_float(o[e]) * keep);
                tmem_st32(tmem + lanes + O_COL + c, o);
              }
              tmem_wait_st();
            }
            const float m_ref = m_used == -INFINITY ? 0.f : m_used;  // none of a copy's tokens is there
            // The reference comes from a rounded product; a fused weight's exponent
            // keeps what was rounded off there, up to half a step.  Of scores FAR out
            // that passes the type's range (fp16's from 2^24 on, bf16's from 2^31
            // on), so there the product is rounded as the maximum's was.
            const bool far = __any_sync(0xFFFFFFFFu, live && fabsf(m_ref) >= FAR);  // (lanes without a row: anything)
            const float factor = far ? 1.f : p.scale_log2;
            if (m >= 2) {
              ok = __all_sync(0xFFFFFFFFu, role_wait(&s->p_free[m & 1], ((m >> 1) - 1) & 1, s, p.status));
              if (!ok) break;
              tc_fence_after();
            }
            const uint32_t pt = tmem + lanes + P_COL + (m & 1) * (TK / 2) + copy * (CW / 2);
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
            for (int c0 = CW - CX; c0 >= 0; c0 -= CX) {
              if (c0 != CW - CX) scores(c0);
              uint32_t w2[CX / 2];
              if (far) {
#pragma unroll
                for (int c = 0; c < CX; c++) x[c] = __fmul_rn(x[c], p.scale_log2);
              }
#pragma unroll
              for (int c = 0; c < CX; c++) x[c] = exp2_approx(fmaf(x[c], factor, -m_ref));
              if (valid < CW) {
#pragma unroll
                for (int c = 0; c < CX; c++)
                  if (c0 + c >= valid) x[c] = 0.f;
              }
#pragma unroll
              for (int c = 0; c < CX; c += 2) {
                sum[(c >> 1) & 3] += x[c] + x[c + 1];
                w2[c / 2] = pack2(x[c], x[c + 1], T());
              }
              if constexpr (CX == 32)
                tmem_st16(pt + c0 / 2, w2);
              else
                tmem_st8(pt + c0 / 2, w2);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s->s_free[m & 1]);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s->p_full[m & 1]);
          }
        }
        if (ok) ok = __all_sync(0xFFFFFFFFu, role_wait(&s->o_full, seg & 1, s, p.status));
        s->m[at] = m_used;
        s->l[at] = l;
        if (!softmax_bar(ok)) {
          if (at == 0) (void)mbar_wait(&s->q_full, seg & 1);  // nothing leaves while its copies are in flight
          break;
        }
        tc_fence_after();
        // the copies' sums on a common maximum, added through the query rows'
        // memory (their product is done), 32 or 64 columns at a time, and
        // written [column][row]: a warp's store is one run
        float top = -INFINITY, total = 0.f;
#pragma unroll
        for (int k = 0; k < SPLIT; k++) top = fmaxf(top, s->m[k * LANES + row]);
#pragma unroll
        for (int k = 0; k < SPLIT; k++) {
          const float mk = s->m[k * LANES + row];
          if (mk != -INFINITY) total += s->l[k * LANES + row] * exp2_approx(mk - top);
        }
        if constexpr (SPLIT > 1) {  // this lane's factor, for the threads that add the copies
          softmax_sync();           // the maxima have been read
          s->m[at] = m_used == -INFINITY ? 0.f : exp2_approx(m_used - top);
          softmax_sync();
        }
        float* item = p.partial + (int64_t)(blockIdx.x + w.b * p.cache.heads + w.h) * (D + 2) * p.Rp;
        float* part = item + row;
        // a lane's columns lie together, their 16-byte units swizzled by the lane
        // (64 at a time where registers allow)
        constexpr int CH = (D == 256 && SPLIT > 1) || (D == 128 && SPLIT == 4) ? 64 : 32, UNITS = CH / 16;  // a thread's own of them
        constexpr int BUFFERS = q_bytes(D) >= 2 * ATT_ROWS * CH * 4 ? 2 : 1;
        uint32_t x[CH];
        auto fetch = [&](int c0) {
#pragma unroll
          for (int c = 0; c < CH; c += 32) tmem_ld32(tmem + lanes + O_COL + c0 + c, x + c);
        };
        constexpr bool EARLY = CH == 32 && SPLIT > 1;  // the next columns on their way during the exchange
        if (EARLY && warp < active) fetch(0);
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += CH) {
          const uint32_t buf = q_smem + c0 / CH % BUFFERS * (ATT_ROWS * CH * 4);
          if (warp < active) {
            if (!EARLY) fetch(c0);
            tmem_wait_ld();
            if constexpr (SPLIT == 1) {
              if (live) {
#pragma unroll
                for (int c = 0; c < CH; c++) part[(c0 + c) * p.Rp] = __uint_as_float(x[c]);
              }
            } else if (live) {
#pragma unroll
              for (int c = 0; c < CH; c += 4)
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(buf + at * (CH * 4) + (((c / 4) ^ (at & 7)) << 4)),
                             "r"(x[c]), "r"(x[c + 1]), "r"(x[c + 2]), "r"(x[c + 3])
                             : "memory");
            }
            if (EARLY && c0 + CH < D) fetch(c0 + CH);
          }
          if constexpr (SPLIT > 1) {
            softmax_sync();
            // CH / 16 columns of every eighth row per thread
            const int r8 = at & 7, c = (at >> 3) * UNITS;
            for (int r = r8; r < p.R; r += 8) {
              float v[UNITS];
#pragma unroll
              for (int e = 0; e < UNITS; e++) v[e] = 0.f;
#pragma unroll
              for (int k = 0; k < SPLIT; k++) {
                const int from = k * LANES + r;  // from & 7 = r8
                const float f = s->m[from];
                const uint32_t a = buf + from * (CH * 4) + (((c >> 2) ^ r8) << 4) + ((c & 2) << 2);
                float y[4];
                if constexpr (UNITS == 4)
                  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                               : "=f"(y[0]), "=f"(y[1]), "=f"(y[2]), "=f"(y[3])
                               : "r"(a)
                               : "memory");
                else
                  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(y[0]), "=f"(y[1]) : "r"(a) : "memory");
#pragma unroll
                for (int e = 0; e < UNITS; e++) v[e] = fmaf(f, y[e], v[e]);
              }
#pragma unroll
              for (int e = 0; e < UNITS; e++) item[(c0 + c + e) * p.Rp + r] = v[e];
            }
            // with two buffers the next chunk's barrier stands between these reads and the writes after it
            if (BUFFERS == 1 && c0 + CH < D) softmax_sync();
          }
        }
        // the next item's query rows may land once all four warps are done
        // with this memory and with O
        fence_proxy_async_smem();
        tc_fence_before();
        softmax_sync();
        if (live && copy == 0) {
          part[D * p.Rp] = top;
          part[(D + 1) * p.Rp] = total;
        }
        n += (uint32_t)w.n;
        seg++;
      } while (next_item<TK, GAP>(p, w));
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == ISSUER) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins an item's partial results with the step's own rows, eight query rows
// and 32 to 128 columns per block: o = (sum_s 2^(m_s - M) O_s + sum_j 2^(x_j - M) v_j)
// / (the same sum of weights).  The scores x_j of the keys that a row sees are
// formed before the first launch is waited for.  A few hundred KB from L2.
template <typename T, int D, int JOIN_COLS>
__global__ void __launch_bounds__(JOIN_THREADS, 2) qlin_attention_join_kernel(const __grid_constant__ AttentionParams p) {
  constexpr int JOIN_GROUPS = JOIN_THREADS / (2 * JOIN_COLS);  // threads that share a column's partial results
  __shared__ __align__(16) float weight[ATT_MAX_CTAS][8];  // of each partial result, per row
  __shared__ float own[QLIN_MAX_TREE][8];                  // of each of the step's rows
  __shared__ int64_t place[QLIN_MAX_TREE];
  __shared__ __align__(16) float sums[JOIN_GROUPS][JOIN_COLS][8];
  __shared__ int64_t range[2];
  constexpr int E = D / 32, TILE = tile_tokens(D);
  const int item = blockIdx.x, b = item / p.cache.heads, h = item % p.cache.heads;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r0 = blockIdx.y * 8, row = r0 + warp, t = row / p.group;
  const int len = p.step.len[b], rows = step_rows(p.step, b);
  const bool live = len >= 0 && warp < 8 && row < p.R && t < rows;  // a warp per row for its weights
  if (warp == 8) {
    int64_t before, all;
    work_before<TILE, GAP>(p, b, &before, &all);
    if (lane == 0) range[0] = before, range[1] = all;
  }
  if (len >= 0 && warp == 0) {
    if (lane < rows) {
      place[lane] = token_offset(p.cache, p.step, b, (int64_t)len + lane);
      if (place[lane] < 0 || (int64_t)len > (int64_t)p.step.max_pages * p.cache.page_size)
        report(p.status, QLIN_ERR_BAD_INDEX);
    }
  }
  __syncthreads();
  float mine = -INFINITY;  // lane j: the score of row j of the step
  if (live) {
    const uint32_t mask = step_mask(p.step, b, t);
    const int64_t head = (int64_t)h * p.group + row % p.group;
    const T* q = static_cast<const T*>(p.q) + ((int64_t)b * p.step.T + t) * p.q_stride + head * D + lane * E;
    float2 f[E / 2];
#pragma unroll
    for (int e = 0; e < E; e += 2) f[e / 2] = unpack2(*reinterpret_cast<const uint32_t*>(q + e), T());
#pragma unroll 4
    for (int j = 0; j < rows; j++) {
      if (!(mask >> j & 1) || place[j] < 0) continue;
      const T* k = static_cast<const T*>(p.cache.k) + place[j] + h * p.cache.head_stride + lane * E;
      float x = 0.f;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float2 g = unpack2(*reinterpret_cast<const uint32_t*>(k + e), T());
        x = fmaf(f[e / 2].x, g.x, fmaf(f[e / 2].y, g.y, x));
      }
#pragma unroll
      for (int i = 16; i; i >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, i);
      if (lane == j) mine = x * p.scale_log2;
    }
  }
  // this item's tiles among all, and the CTAs whose runs hold them
  const int64_t per = tokens_to_tiles<TILE>(p.tokens(b)), N = range[1];
  const int64_t start = range[0] + h * (per + GAP);
  const int runs = runs_of(p, N);
  const int first = per ? cta_of(start, N, runs) : 0;
  const int parts = per ? cta_of(start + per - 1, N, runs) - first + 1 : 0;
  // four rows and a column per thread, every JOIN_GROUPS-th partial result and row of the step
  const int half = threadIdx.x & 1, c = (threadIdx.x >> 1) % JOIN_COLS, group = threadIdx.x / (2 * JOIN_COLS);
  const int col = blockIdx.z * JOIN_COLS + c;
  uint32_t mask[4];
#pragma unroll
  for (int k = 0; k < 4; k++) {
    const int r = r0 + half * 4 + k, tr = r / p.group;
    mask[k] = len >= 0 && r < p.R && tr < rows ? step_mask(p.step, b, tr) : 0;
  }
  const uint32_t any = mask[0] | mask[1] | mask[2] | mask[3];
  auto own_value = [&](int j) -> float {
    if (j >= rows || !(any >> j & 1) || place[j] < 0) return 0.f;
    return to_float(static_cast<const T*>(p.cache.v)[place[j] + h * p.cache.head_stride + col]);
  };
  constexpr int EARLY = 2;  // of a thread's rows of the step, those whose value is read before the wait
  float y[EARLY];
#pragma unroll
  for (int i = 0; i < EARLY; i++) y[i] = own_value(group + i * JOIN_GROUPS);
  const uint32_t seen_mask = live ? step_mask(p.step, b, t) : 0;
  pdl_wait();
  pdl_launch_dependents();
  if (len < 0 || rows == 0) return;
  const int64_t step = (int64_t)(D + 2) * p.Rp;
  const float* part = p.partial + (int64_t)(first + item) * step + r0;
  // the first partial results are on their way while the weights are formed
  constexpr int AHEAD = 6;
  const float4* x = reinterpret_cast<const float4*>(part + (int64_t)col * p.Rp + half * 4);
  float4 early[AHEAD];
#pragma unroll
  for (int k = 0; k < AHEAD; k++)
    if (group + k * JOIN_GROUPS < parts) early[k] = x[(group + k * JOIN_GROUPS) * (step / 4)];
  if (live) {
    constexpr int PER = (ATT_MAX_CTAS + 31) / 32;
    float pm[PER], pl[PER], m = mine;
#pragma unroll
    for (int k = 0; k < PER; k++) {
      const float* ml = part + (lane + 32 * k) * step + (int64_t)D * p.Rp + warp;
      const bool there = lane + 32 * k < parts;
      pm[k] = there ? ml[0] : -INFINITY;
      pl[k] = there ? ml[p.Rp] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < PER; k++) m = fmaxf(m, pm[k]);
#pragma unroll
    for (int i = 16; i; i >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, i));
    const bool seen = lane < rows && (seen_mask >> lane & 1) && place[lane] >= 0;
    const float w = seen ? exp2f(mine - m) : 0.f;
    float l = w;
#pragma unroll
    for (int k = 0; k < PER; k++) {
      pm[k] = lane + 32 * k < parts ? exp2f(pm[k] - m) : 0.f;
      l = fmaf(pm[k], pl[k], l);
    }
#pragma unroll
    for (int i = 16; i; i >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, i);
    if (p.stats && blockIdx.z == 0 && lane == 0)
      reinterpret_cast<float2*>(p.stats)[((int64_t)b * p.step.T + t) * ((int64_t)p.group * p.cache.heads) +
                                         (int64_t)h * p.group + row % p.group] = make_float2(m, l);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    own[lane][warp] = w * inv;
#pragma unroll
    for (int k = 0; k < PER; k++)
      if (lane + 32 * k < parts) weight[lane + 32 * k][warp] = pm[k] * inv;
  }
  __syncthreads();
  {
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](int i, const float4& v) {
      const float4 f = *reinterpret_cast<const float4*>(&weight[i][half * 4]);
      acc.x = fmaf(f.x, v.x, acc.x), acc.y = fmaf(f.y, v.y, acc.y);
      acc.z = fmaf(f.z, v.z, acc.z), acc.w = fmaf(f.w, v.w, acc.w);
    };
#pragma unroll
    for (int k = 0; k < AHEAD; k++)
      if (group + k * JOIN_GROUPS < parts) add(group + k * JOIN_GROUPS, early[k]);
    for (int i0 = group + AHEAD * JOIN_GROUPS; i0 < parts; i0 += AHEAD * JOIN_GROUPS) {
      float4 v[AHEAD];
#pragma unroll
      for (int k = 0; k < AHEAD; k++)
        if (i0 + k * JOIN_GROUPS < parts) v[k] = x[(i0 + k * JOIN_GROUPS) * (step / 4)];
#pragma unroll
      for (int k = 0; k < AHEAD; k++)
        if (i0 + k * JOIN_GROUPS < parts) add(i0 + k * JOIN_GROUPS, v[k]);
    }
    auto add_own = [&](int j, float value) {  // only what a row sees: what it does not may be NaN
      const float* f = &own[j][half * 4];
      if (mask[0] >> j & 1) acc.x = fmaf(f[0], value, acc.x);
      if (mask[1] >> j & 1) acc.y = fmaf(f[1], value, acc.y);
      if (mask[2] >> j & 1) acc.z = fmaf(f[2], value, acc.z);
      if (mask[3] >> j & 1) acc.w = fmaf(f[3], value, acc.w);
    };
#pragma unroll
    for (int i = 0; i < EARLY; i++)
      if (group + i * JOIN_GROUPS < rows && place[group + i * JOIN_GROUPS] >= 0) add_own(group + i * JOIN_GROUPS, y[i]);
#pragma unroll 4
    for (int j = group + EARLY * JOIN_GROUPS; j < rows; j += JOIN_GROUPS)
      if (place[j] >= 0) add_own(j, own_value(j));
    *reinterpret_cast<float4*>(&sums[group][c][half * 4]) = acc;
  }
  __syncthreads();
  if (live) {  // a row's columns: one run
    __nv_bfloat16* out = p.out + ((int64_t)b * p.step.T + t) * p.out_stride +
                         ((int64_t)h * p.group + row % p.group) * D + blockIdx.z * JOIN_COLS;
#pragma unroll
    for (int e = lane; e < JOIN_COLS; e += 32) {
      float o = 0.f;
#pragma unroll
      for (int g = 0; g < JOIN_GROUPS; g++) o += sums[g][e][warp];
      out[e] = __float2bfloat16(o);
    }
  }
}

struct Kernels {
  const void *main[3], *join[3];  // main: 1, 2 and 4 copies of the query rows; join: 32, 64 and (from width 128) 128 columns
};
template <typename T, int D>
Kernels kernels_of() {
  return {{reinterpret_cast<const void*>(qlin_attention_kernel<T, D, 1>),
           reinterpret_cast<const void*>(qlin_attention_kernel<T, D, 2>),
           reinterpret_cast<const void*>(qlin_attention_kernel<T, D, 4>)},
          {reinterpret_cast<const void*>(qlin_attention_join_kernel<T, D, 32>),
           reinterpret_cast<const void*>(qlin_attention_join_kernel<T, D, 64>),
           reinterpret_cast<const void*>(qlin_attention_join_kernel<T, D, (D < 128 ? 64 : 128)>)}};
}
Kernels attention_kernels(int dtype, int width) {
  if (dtype == QLIN_BF16)
    return width == 64    ? kernels_of<__nv_bfloat16, 64>()
           : width == 128 ? kernels_of<__nv_bfloat16, 128>()
                          : kernels_of<__nv_bfloat16, 256>();
  return width == 64 ? kernels_of<__half, 64>() : width == 128 ? kernels_of<__half, 128>() : kernels_of<__half, 256>();
}
// A test's: bf16 of width 128, up to 32 query rows of a cache head.
const void* attention_fault_kernel() {
  return reinterpret_cast<const void*>(qlin_attention_kernel<__nv_bfloat16, 128, 4, true>);
}
constexpr size_t attention_smem(int width) {  // query rows, ring, and the way to a 1024-byte boundary
  return (size_t)q_bytes(width) + (size_t)ring_buffers(width) * tile_bytes(width) + 1024;
}

struct AttentionDevice {
  std::once_flag once;
  qlin_status ready = QLIN_ERR_CUDA;
  int ctas = 0;
};
AttentionDevice g_attention[64];

// SM count, kernel attributes and the driver's encoder, once per device.
qlin_status attention_setup(int* ctas) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return status_of(e);
  if (dev < 0 || dev >= 64) return QLIN_ERR_CUDA;
  AttentionDevice& d = g_attention[dev];
  std::call_once(d.once, [&d, dev] {
    int sms = 0;
    cudaError_t e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    auto prepare = [&e](const void* fn, int width) {
      for (auto set : {std::make_pair(cudaFuncAttributeMaxDynamicSharedMemorySize, (int)attention_smem(width)),
                       // all of it as shared memory, so that the second launch's blocks fit beside
                       std::make_pair(cudaFuncAttributePreferredSharedMemoryCarveout, (int)cudaSharedmemCarveoutMaxShared)})
        if (e == cudaSuccess) e = cudaFuncSetAttribute(fn, set.first, set.second);
    };
    for (int dtype : {QLIN_BF16, QLIN_F16})
      for (int width : {64, 128, 256})
        for (const void* fn : attention_kernels(dtype, width).main) prepare(fn, width);
    prepare(attention_fault_kernel(), 128);
    d.ctas = sms < ATT_MAX_CTAS ? sms : ATT_MAX_CTAS;
    d.ready = e == cudaSuccess && encode_tiled() && sms > 0 ? QLIN_OK : QLIN_ERR_CUDA;
    if (e != cudaSuccess) (void)cudaGetLastError();
  });
  *ctas = d.ctas;
  return d.ready;
}

// The query rows [B * T, Hq, width] as boxes of 64 elements x group x T: an
// item's rows in order, row t * group + i
bool encode_q(CUtensorMap* map, const qlin_kv_cache* c, const qlin_kv_step* s, const void* q, int64_t stride, int Hq) {
  const cuuint64_t dims[3] = {(cuuint64_t)c->width, (cuuint64_t)Hq, (cuuint64_t)((int64_t)s->B * s->T)};
  const cuuint64_t strides[2] = {(cuuint64_t)c->width * 2, (cuuint64_t)stride * 2};
  const cuuint32_t shape[3] = {64, (cuuint32_t)(Hq / c->heads), (cuuint32_t)s->T}, one[3] = {1, 1, 1};
  return encode_tiled()(map, c->dtype == QLIN_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                  const_cast<void*>(q), dims, strides, shape, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

qlin_status check_heads(const qlin_kv_cache* c, int64_t B, int64_t T, int Hq) {
  if (B < 0 || T < 0 || Hq < 1 || Hq % c->heads) return QLIN_ERR_INVALID_ARG;
  if (T > QLIN_MAX_TREE || T * (Hq / c->heads) > ATT_ROWS) return QLIN_ERR_UNSUPPORTED;
  if (B * c->heads > (1 << 24)) return QLIN_ERR_UNSUPPORTED;
  return QLIN_OK;
}
int padded_rows(int64_t T, int group) { return (int)((T * group + 7) / 8 * 8); }

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
  // a part of an item ends where the item or a CTA's run ends
  const size_t slots = ATT_MAX_CTAS + (size_t)B * cache->heads;
  *bytes = (size_t)STEP_WS_HEADER + slots * (cache->width + 2) * padded_rows(T, Hq / cache->heads) * sizeof(float);
  return QLIN_OK;
}

static qlin_status attend(const qlin_kv_cache* cache, const qlin_kv_step* step, int Hq, const void* q, int64_t q_stride,
                          float scale, void* out, int64_t out_stride, void* ws, size_t ws_bytes, unsigned flags,
                          void* stream, float* stats, int64_t fault_copy = -1) {
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
  // the second launch writes some columns of a row while others read its q
  if (rows_overlap(out, out_stride * 2, Hq * D * 2, q, q_stride * 2, Hq * D * 2, (int64_t)step->B * step->T))
    return QLIN_ERR_INVALID_ARG;
  if (stats) {  // written where other blocks still read q
    const int64_t n = (int64_t)step->B * step->T;
    if (!is_aligned(stats, 8) || rows_overlap(stats, Hq * 8, Hq * 8, q, q_stride * 2, Hq * D * 2, n) ||
        rows_overlap(stats, Hq * 8, Hq * 8, out, out_stride * 2, Hq * D * 2, n))
      return QLIN_ERR_INVALID_ARG;
  }
  int ctas = 0;
  st = attention_setup(&ctas);
  if (st != QLIN_OK) return st;
  AttentionParams p;
  const int tile = tile_tokens(cache->width);
  p.box = cache->page_size < tile ? cache->page_size : tile;
  if (!encode(encode_tiled(), &p.map_k, cache, cache->k, p.box) || !encode(encode_tiled(), &p.map_v, cache, cache->v, p.box) ||
      !encode_q(&p.map_q, cache, step, q, q_stride, Hq))
    return QLIN_ERR_CUDA;
  p.page_shift = 0;
  while ((1 << p.page_shift) < cache->page_size) p.page_shift++;
  p.cache = *cache;
  p.step = *step;
  p.q = q;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.q_stride = q_stride, p.out_stride = out_stride;
  p.status = static_cast<uint32_t*>(ws);
  p.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + STEP_WS_HEADER);
  p.scale_log2 = (float)((double)scale * 1.4426950408889634);
  p.group = Hq / cache->heads;
  p.R = step->T * p.group;
  p.Rp = padded_rows(step->T, p.group);
  p.ctas = ctas;
  p.fault_copy = fault_copy;
  p.stats = stats;
  void* args[] = {&p};
  const Kernels fn = attention_kernels(cache->dtype, cache->width);
  const int copies = p.R > ATT_ROWS / 2 ? 0 : p.R > ATT_ROWS / 4 ? 1 : 2;
  const void* const main = fault_copy < 0 ? fn.main[copies] : attention_fault_kernel();
  st = launch_step(main, dim3((unsigned)ctas, 1, 1), dim3(ATT_THREADS, 1, 1), attention_smem(cache->width),
                   static_cast<cudaStream_t>(stream), args, (flags & QLIN_FLAG_PDL) != 0);
  if (st != QLIN_OK) return st;
  // the narrowest blocks that all find room while the first launch runs, one
  // per SM: more of them would start behind it
  const int64_t blocks = (int64_t)step->B * cache->heads * (p.Rp / 8);
  int wide = 0;
  while (wide < (D < 128 ? 1 : 2) && blocks * (D / (32 << wide)) > ctas) wide++;
  return launch_step(fn.join[wide], dim3((unsigned)(step->B * cache->heads), (unsigned)(p.Rp / 8), (unsigned)(D / (32 << wide))),
                     dim3(JOIN_THREADS, 1, 1), 0, static_cast<cudaStream_t>(stream), args, true);
}

qlin_status qlin_tree_attention(const qlin_kv_cache* cache, const qlin_kv_step* step, int Hq, const void* q,
                                int64_t q_stride, float scale, void* out, int64_t out_stride, void* ws,
                                size_t ws_bytes, unsigned flags, void* stream) {
  return attend(cache, step, Hq, q, q_stride, scale, out, out_stride, ws, ws_bytes, flags, stream, nullptr);
}

qlin_status qlin_tree_attention_stats(const qlin_kv_cache* cache, const qlin_kv_step* step, int Hq, const void* q,
                                      int64_t q_stride, float scale, void* out, int64_t out_stride, float* stats,
                                      void* ws, size_t ws_bytes, unsigned flags, void* stream) {
  if (!stats && (!step || (step->B != 0 && step->T != 0))) return QLIN_ERR_INVALID_ARG;
  return attend(cache, step, Hq, q, q_stride, scale, out, out_stride, ws, ws_bytes, flags, stream, stats);
}

qlin_status qlin_debug_tree_attention_fault(const qlin_kv_cache* cache, const qlin_kv_step* step, int Hq,
                                            const void* q, int64_t q_stride, float scale, void* out,
                                            int64_t out_stride, void* ws, size_t ws_bytes, int64_t copy,
                                            void* stream) {
  const qlin_status st = check_cache(cache);
  if (st != QLIN_OK) return st;
  if (copy < 0 || !step || step->T < 0 || Hq < 1) return QLIN_ERR_INVALID_ARG;
  if (cache->dtype != QLIN_BF16 || cache->width != 128 || (int64_t)step->T * (Hq / cache->heads) > ATT_ROWS / 4)
    return QLIN_ERR_UNSUPPORTED;
  return attend(cache, step, Hq, q, q_stride, scale, out, out_stride, ws, ws_bytes, 0, stream, nullptr, copy);
}

}  // extern "C"
