// qlin_kv_weigh: the attention weight that each cached token got from a step's
// rows, added to what it got before.
#include <cmath>
#include <mutex>
#include <type_traits>

#include "qlin_tiles.cuh"

namespace qlin {
namespace {

constexpr int SETS = 4;             // of four weighing warps each, which take the tiles in turn
constexpr int PRODUCERS = 2;        // warps that load tiles in turn
constexpr int PRODUCER = 4 * SETS, ISSUER = PRODUCER + PRODUCERS;
constexpr int WEIGHING = 128 * SETS, WEIGH_THREADS = WEIGHING + 32 * PRODUCERS + 32;
constexpr int TILE = 128;           // tokens of a tile: the lanes of tensor memory
constexpr int MAX_ROWS = 128;       // query rows of an item at most: columns of an accumulator
constexpr int SLOT_BYTES = TILE * 128;  // a ring slot: a 64-wide panel of a tile's keys
constexpr int MAX_SLOTS = 12, ACCUMULATORS = 4;
constexpr int WEIGH_SMEM = 208 * 1024;
constexpr int GAP = 1;              // work of a change to another item, in tiles
constexpr uint32_t ALL = 0xFFFFFFFFu;
constexpr float FAR = 0x1p23f;      // from here on fp32 scores (log2 units) are a step or more apart

struct WeighParams {
  CUtensorMap map_k;
  qlin_kv_cache cache;
  qlin_kv_step step;
  const void* q;
  const float2* stats;
  const int32_t *keep, *n_keep, *at;
  const float* score;
  float* score_out;
  int32_t* position_out;
  int64_t q_stride, keep_stride, seq_stride, head_stride, out_seq_stride, out_head_stride;
  uint32_t* status;
  float scale_log2, decay;
  int room;
  uint32_t group_inverse;  // 2^16 / group, rounded up: the kept row of a column (below 128)
  int group, Rp;   // query heads of a cache head; columns of an accumulator: T * group, padded to 16
  int slots;       // of the ring
  int ctas, box, page_shift;
  int64_t fault_copy;  // test only (FAULT): the panel that the first CTA never loads

  // the committed ones that are there and the step's rows
  __device__ __forceinline__ int64_t tokens(int b) const {
    const int64_t len = step.len[b];
    if (len < 0) return 0;
    const int64_t most = (int64_t)step.max_pages * cache.page_size, n = len + step_rows(step, b);
    return n < most ? n : most;
  }
};

struct WeighShared {
  uint64_t full[MAX_SLOTS], empty[MAX_SLOTS], acc_full[ACCUMULATORS], acc_free[ACCUMULATORS], q_full, drained;
  uint32_t tmem;
  int dead;  // a wait has expired: every role leaves its loop
  Walk walk;
  // of the item: two columns' negative references and inverse sums of weights at a time
  float4 stat[MAX_ROWS / 2];
  int kept[QLIN_MAX_TREE];       // the kept rows
  int own[QLIN_MAX_TREE];        // the step's row: its place among the kept ones, or -1
  uint32_t seen[QLIN_MAX_TREE];  // kept rows (bits) that see the step's row
  int rows, far;
};

__device__ __forceinline__ bool role_wait(uint64_t* bar, uint32_t parity, WeighShared* s, uint32_t* status) {
  if (mbar_try_wait(bar, parity)) return true;
  if (!*(volatile int*)&s->dead && mbar_wait(bar, parity)) return true;
  s->dead = 1;
  report(status, QLIN_ERR_DEVICE_TIMEOUT);
  return false;
}
// A barrier of the weighing warps that tells whether all are still at work.
__device__ __forceinline__ bool weighing_bar(bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.and.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"((uint32_t)ok), "n"(WEIGHING)
      : "memory");
  return all != 0;
}
// a * b + c on two numbers
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

// The item's rows and what they see, by one warp.
__device__ __forceinline__ void item_rows(const WeighParams& p, int b, WeighShared* s) {
  const int lane = threadIdx.x & 31, len = p.step.len[b], rows = step_rows(p.step, b);
  s->own[lane] = -1;
  s->seen[lane] = 0;
  __syncwarp();
  int n = rows;
  if (p.keep) {  // an accepted path: each row sees those before it
    n = p.n_keep[b];
    bool bad = n < 0 || n > rows;
    if (bad) n = 0;
    const int r = lane < n ? p.keep[b * p.keep_stride + lane] : 0x7FFFFFFF;
    const int before = __shfl_up_sync(0xFFFFFFFFu, r, 1);
    if (lane < n && (r < 0 || r >= rows || (lane && r <= before))) bad = true;
    if (__any_sync(0xFFFFFFFFu, bad)) {
      if (lane == 0) report(p.status, QLIN_ERR_BAD_INDEX);
      n = 0;
    }
    if (lane < n) {
      s->kept[lane] = r;
      s->own[r] = lane;
      s->seen[r] = (0xFFFFFFFFu >> (32 - n)) & ~((1u << lane) - 1);
    }
  } else {
    const uint32_t mask = lane < n ? step_mask(p.step, b, lane) : 0;
    for (int r = 0; r < n; r++) {
      const uint32_t who = __ballot_sync(0xFFFFFFFFu, mask >> r & 1);
      if (lane == r) s->seen[r] = who;
    }
    if (lane < n) s->kept[lane] = lane, s->own[lane] = lane;
  }
  __syncwarp();
  if (lane == 0) {
    s->rows = n, s->far = 0;
    // committed tokens and kept rows' own behind the table are left out
    if (len + (int64_t)(n ? s->kept[n - 1] + 1 : 0) > (int64_t)p.step.max_pages * p.cache.page_size)
      report(p.status, QLIN_ERR_BAD_INDEX);
  }
}

// X = K Q^T on tcgen05, a tile of 128 tokens as the rows (lanes of tensor memory)
// and the query rows as the columns, so that a thread owns a token and adds up its
// weights sum_r 2^(c x_r - reference_r) / l_r in registers, without an exchange.
// Keys come by TMA in panels of 64 columns (128-byte swizzle), read by the tensor
// cores from the ring; the query rows lie in shared memory for an item's length.
// Items are cut into equal runs as in tree attention.  Four accumulators, and as
// many sets of weighing warps, so that a tile's latencies (tensor memory to
// registers, exponentials, the score's way back) are hidden by three others.
//
// Bound by the stream of keys: 32 KB of a tile take an SM 0.74 us at the measured
// copy bandwidth.  Measured: one row of 6 heads over 131k tokens of 8 heads of 128,
// 48.0 us for 277 MB (0.85 of the copy; the rest is the start: length, page table,
// first keys); 96 rows 48.9 us (0.84); up to 30 rows over 8 sequences of up to 30011
// tokens, 342 MB, 60.0 us (0.84); one token's rows over 1777 tokens 7.0 us, the
// chain of dependent reads before the first keys.  With two sets and one producer
// the 96 rows took 65.7 us with pages of 16.
template <typename T, int D, bool FAULT = false>
__global__ void __launch_bounds__(WEIGH_THREADS, 1) qlin_weigh_kernel(const __grid_constant__ WeighParams p) {
  extern __shared__ uint8_t raw[];
  __shared__ WeighShared sh;
  WeighShared* s = &sh;
  constexpr int PANELS = D / 64;
  const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
  const uint32_t panel_bytes = (uint32_t)p.Rp * 128, q_smem = base, ring = base + PANELS * panel_bytes;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.slots; i++) mbar_init(&s->full[i], 1), mbar_init(&s->empty[i], 1);
    for (int i = 0; i < ACCUMULATORS; i++) mbar_init(&s->acc_full[i], 1), mbar_init(&s->acc_free[i], 4);
    mbar_init(&s->q_full, 1);
    mbar_init(&s->drained, 1);
    s->dead = 0;
    mbar_fence_init();
  }
  if (warp == ISSUER) tmem_alloc(&s->tmem, 512);
  pdl_wait();
  pdl_launch_dependents();
  if (warp == PRODUCER) {
    const Walk w = first_item<TILE, GAP>(p, blockIdx.x);
    if (lane == 0) s->walk = w;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s->tmem;
  Walk w = s->walk;

  if (w.left > 0) {
    if (warp >= PRODUCER && warp < ISSUER) {
      // ---- a lane per TMA copy (a page's or a tile's rows of a panel), the
      // producers' warps a tile each in turn: a warp's lanes issue their copies one
      // after the other, of small pages too slowly for the memory
      const int copies = TILE / p.box, box = lane % copies, panel = lane / copies;  // at most 8 and 4
      const uint32_t slots = (uint32_t)p.slots, mine = (uint32_t)(warp - PRODUCER);
      uint32_t i = mine * PANELS + panel, slot = i, phase = 1;  // this lane's next panel of the run, its place in the ring
      uint32_t n = 0;                                           // tiles of the items before
      bool ok = true;
      do {
        const int32_t* table = p.step.page_table + w.b * p.step.table_stride;
        const int skip = (int)((mine + PRODUCERS - n % PRODUCERS) % PRODUCERS);  // tiles of the item before this warp's first
        int64_t token = (w.tile + skip) * TILE + box * p.box;
        auto page_of = [&](int64_t t, int64_t at) { return t < w.n && panel < PANELS && at < w.tokens ? table[at >> p.page_shift] : -1; };
        int next = page_of(skip, token);
        for (int64_t t = skip; t < w.n && ok; t += PRODUCERS, token += PRODUCERS * TILE) {
          int page = next;
          if (panel < PANELS && token < w.tokens && (page < 0 || page >= p.cache.pages)) {
            page = -1;
            report(p.status, QLIN_ERR_BAD_INDEX);
          }
          next = page_of(t + PRODUCERS, token + PRODUCERS * TILE);
          if (i >= slots && panel < PANELS) ok = role_wait(&s->empty[slot], phase, s, p.status);
          ok = __all_sync(ALL, ok);
          if (!ok) break;
          const uint32_t bytes = __popc(__ballot_sync(ALL, page >= 0 && panel == 0)) * p.box * 128;
          if (box == 0 && panel < PANELS) mbar_arrive_expect_tx(&s->full[slot], bytes);
          __syncwarp();
          const bool lost = FAULT && blockIdx.x == 0 && i == p.fault_copy;  // test only: never completes
          if (page >= 0 && !lost)
            tma_load_4d(ring + slot * SLOT_BYTES + box * p.box * 128, &p.map_k, panel * 64,
                        (int)(token & (p.cache.page_size - 1)), w.h, page, &s->full[slot]);
          i += PRODUCERS * PANELS;
          slot += PRODUCERS * PANELS;
          if (slot >= slots) slot -= slots, phase ^= 1;
        }
        n += (uint32_t)w.n;
      } while (ok && next_item<TILE, GAP>(p, w));
      // nothing leaves while its copies are in flight, whichever role gave up: of
      // the ring's last round, as what lies before that has been waited for
      const uint32_t end = ok ? n * PANELS : i;
      if (box == 0 && panel < PANELS)
        for (uint32_t j = i; j >= PRODUCERS * PANELS;) {
          j -= PRODUCERS * PANELS;
          if (j + slots < end) break;
          (void)mbar_wait(&s->full[j % slots], j / slots & 1);
        }
    } else if (warp == ISSUER) {
      constexpr uint32_t type = std::is_same<T, __nv_bfloat16>::value ? (1u << 7) | (1u << 10) : 0u;
      const uint32_t id = mma_idesc_f16(TILE, p.Rp) | type;
      uint32_t m = 0, seg = 0, slot = 0, phase = 0;
      bool ok = true;
      do {
        ok = __all_sync(0xFFFFFFFFu, role_wait(&s->q_full, seg & 1, s, p.status));
        const int tiles = __shfl_sync(0xFFFFFFFFu, (int)w.n, 0);
        for (int t = 0; t < tiles && ok; t++, m++) {
          const uint32_t acc = m % ACCUMULATORS, d = tmem + acc * MAX_ROWS;
          if (m >= ACCUMULATORS)
            ok = __all_sync(ALL, role_wait(&s->acc_free[acc], (m / ACCUMULATORS - 1) & 1, s, p.status));
          for (int e = 0; e < PANELS && ok; e++) {
            ok = __all_sync(0xFFFFFFFFu, role_wait(&s->full[slot], phase, s, p.status));
            if (!ok) break;
            tc_fence_after();
            const uint32_t at = __shfl_sync(0xFFFFFFFFu, slot, 0), kb = ring + at * SLOT_BYTES, qb = q_smem + e * panel_bytes;
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < 4; k++)
                mma_smem_a(d, swizzled_desc(kb + k * 32, 16), swizzled_desc(qb + k * 32, 16), id, e > 0 || k > 0);
              mma_commit(&s->empty[at]);
              if (e == PANELS - 1) mma_commit(&s->acc_full[acc]);
            }
            __syncwarp();
            if (++slot == (uint32_t)p.slots) slot = 0, phase ^= 1;
          }
        }
        seg++;
      } while (ok && next_item<TILE, GAP>(p, w));
      // whichever role gave up, the products in flight end before tensor memory is freed
      if (__any_sync(ALL, !ok || *(volatile int*)&s->dead) && elect_one()) {
        mma_commit(&s->drained);
        (void)mbar_wait(&s->drained, 0);
      }
    } else if (warp < PRODUCER) {
      // ---- weighing: sets of four warps take the tiles in turn
      const int tid = threadIdx.x, set = warp / 4;
      const int at = tid % TILE;  // this thread's token of a tile
      const uint32_t lanes = (uint32_t)(warp % 4 * 32) << 16;
      uint32_t m = 0;
      bool ok = true;
      do {
        // the item's rows, once all tiles of the one before have been weighed
        if (!weighing_bar(ok)) break;
        if (warp == 0) item_rows(p, w.b, s);
        weighing_bar(true);
        const int n = s->rows, cols = n * p.group;
        const int64_t row0 = (int64_t)w.b * p.step.T;
        static_assert(WEIGHING >= MAX_ROWS, "a thread per column");
        float2 rl = make_float2(0.f, 0.f);  // a column that weighs nothing
        if (tid < cols)
          rl = p.stats[(row0 + s->kept[tid / p.group]) * ((int64_t)p.group * p.cache.heads) + w.h * p.group + tid % p.group];
        // the query rows, swizzled as the keys are by TMA: a thread's units of 16 bytes
        // (the same place of every STEP-th row) all on their way at once
        constexpr int UNITS = D / 8, STEP = WEIGHING / UNITS, MOST = MAX_ROWS / STEP;
        const int u = tid % UNITS;
        auto put = [&](int c, uint4 x) {
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(q_smem + (u / 8) * panel_bytes + c * 128 +
                                                                        (((u & 7) ^ (c & 7)) << 4)),
                       "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w)
                       : "memory");
        };
        uint4 v[MOST];
#pragma unroll
        for (int k = 0; k < MOST; k++) {
          const int c = tid / UNITS + k * STEP;
          v[k] = make_uint4(0, 0, 0, 0);
          if (c < cols)
            v[k] = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) + (row0 + s->kept[c / p.group]) * p.q_stride +
                                                   (int64_t)(w.h * p.group + c % p.group) * D + u * 8);
        }
        // a row that saw nothing, or whose softmax is NaN by a key or a query that is not finite, weighs nothing
        const bool weighs = rl.y > 0.f && rl.y < INFINITY && fabsf(rl.x) < INFINITY;
        if (tid < p.Rp) {
          float* st = reinterpret_cast<float*>(&s->stat[tid / 2]) + tid % 2;
          st[0] = weighs ? -rl.x : -INFINITY;
          st[2] = weighs ? 1.f / rl.y : 0.f;
          if (weighs && fabsf(rl.x) >= FAR) s->far = 1;
        }
#pragma unroll
        for (int k = 0; k < MOST; k++) {
          const int c = tid / UNITS + k * STEP;
          if (c < p.Rp) put(c, v[k]);
        }
        fence_proxy_async_smem();
        // (its query becomes zeros: one that is not finite would reach every token)
        if (!weighing_bar(weighs || tid >= cols)) {
          for (int c = tid / UNITS; c < cols; c += STEP) {
            const float4 st = s->stat[c / 2];
            if ((c & 1 ? st.w : st.z) == 0.f) put(c, make_uint4(0, 0, 0, 0));
          }
          fence_proxy_async_smem();
          weighing_bar(true);
        }
        if (tid == 0) mbar_arrive(&s->q_full);
        const bool far = s->far != 0;
        const int64_t len = p.step.len[w.b];
        const float* score = p.score + w.b * p.seq_stride + w.h * p.head_stride;
        float* score_out = p.score_out + w.b * p.out_seq_stride + w.h * p.out_head_stride;
        int32_t* position_out = p.position_out ? p.position_out + w.b * p.out_seq_stride + w.h * p.out_head_stride : nullptr;
        const int32_t* table = p.step.page_table + w.b * p.step.table_stride;

        for (int t = 0; t < (int)w.n; t++, m++) {
          if ((int)(m % SETS) != set) continue;
          const int64_t first = (w.tile + t) * TILE, token = first + at;
          const bool old = token < len && token < w.tokens;
          const int r = old || token >= w.tokens ? -1 : (int)(token - len), place = r >= 0 ? s->own[r] : -1;
          const int64_t to = place >= 0 ? len + place : token;
          const bool known = (old || place >= 0) && to < p.room;
          if ((old || place >= 0) && to >= p.room) report(p.status, QLIN_ERR_BAD_INDEX);
          const int page = known ? table[token >> p.page_shift] : -1;
          const float before = old && known ? score[token] : 0.f;
          const uint32_t acc = m % ACCUMULATORS;
          ok = __all_sync(0xFFFFFFFFu, role_wait(&s->acc_full[acc], m / ACCUMULATORS & 1, s, p.status));
          if (!ok) break;
          tc_fence_after();
          const uint32_t from = tmem + lanes + acc * MAX_ROWS;
          float2 sum[4] = {};
          const uint32_t seen = old ? ALL : place >= 0 ? s->seen[r] : 0;  // of the kept rows
          if (!far) {
            uint32_t x[32];  // 32 columns at a time
            const float2 scale = make_float2(p.scale_log2, p.scale_log2);
            auto weights = [&](int c, const float4& st) {  // of two columns, but for the sums of weights
              const float2 e = fma2(make_float2(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), scale, make_float2(st.x, st.y));
              return make_float2(exp2_approx(e.x), exp2_approx(e.y));
            };
            auto add = [&](int c0, int c, auto every) {
              const float4 st = s->stat[(c0 + c) / 2];
              float2 e = weights(c, st);
              if constexpr (!decltype(every)::value) {  // what a row does not see may be NaN
                if (!(seen >> ((c0 + c) * p.group_inverse >> 16) & 1)) e.x = 0.f;
                if (!(seen >> ((c0 + c + 1) * p.group_inverse >> 16) & 1)) e.y = 0.f;
              }
              sum[c / 2 & 3] = fma2(e, make_float2(st.z, st.w), sum[c / 2 & 3]);
            };
            auto all = [&](auto every) {
#pragma unroll 1
              for (int c0 = 0; c0 < p.Rp; c0 += 32) {
                const bool half = p.Rp - c0 < 32;
                if (half)
                  tmem_ld16(from + c0, *reinterpret_cast<uint32_t(*)[16]>(x));
                else
                  tmem_ld32(from + c0, x);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 16; c += 2) add(c0, c, every);
                if (half) break;
#pragma unroll
                for (int c = 16; c < 32; c += 2) add(c0, c, every);
              }
            };
            if (first + TILE <= len)  // every row sees every token
              all(std::true_type());
            else
              all(std::false_type());
          } else {
            // A reference far out comes from a rounded product: the scores are rounded
            // as it was, and what still rises above it is no more than a whole weight.
#pragma unroll 1
            for (int c0 = 0; c0 < cols; c0 += 16) {
              uint32_t x[16];
              tmem_ld16(from + c0, x);
              tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < 16; c++)
                if (c0 + c < cols && seen >> ((c0 + c) * p.group_inverse >> 16) & 1) {
                  const float4 st = s->stat[(c0 + c) / 2];
                  const float shift = c & 1 ? st.y : st.x, inv = c & 1 ? st.w : st.z;
                  const float e = exp2_approx(__fmul_rn(__uint_as_float(x[c]), p.scale_log2) + shift) * inv;
                  sum[c & 3].x += e > 1.f ? 1.f : e;
                }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s->acc_free[acc]);
          const float weight = ((sum[0].x + sum[0].y) + (sum[1].x + sum[1].y)) + ((sum[2].x + sum[2].y) + (sum[3].x + sum[3].y));
          if (page >= 0 && page < p.cache.pages) {  // (of one out of range the ring holds another tile's keys)
            score_out[to] = old ? fmaf(p.decay, before, weight) : weight;
            if (!old && position_out) {
              const int64_t row = row0 + r;
              position_out[to] = p.at ? p.at[row]
                                      : (int)len + (p.step.depth ? p.step.depth[w.b * p.step.tree_stride + r] : r);
            }
          }
        }
      } while (next_item<TILE, GAP>(p, w));
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

const void* weigh_fn(int dtype, int width) {
  if (dtype == QLIN_BF16)
    return width == 64    ? reinterpret_cast<const void*>(qlin_weigh_kernel<__nv_bfloat16, 64>)
           : width == 128 ? reinterpret_cast<const void*>(qlin_weigh_kernel<__nv_bfloat16, 128>)
                          : reinterpret_cast<const void*>(qlin_weigh_kernel<__nv_bfloat16, 256>);
  return width == 64    ? reinterpret_cast<const void*>(qlin_weigh_kernel<__half, 64>)
         : width == 128 ? reinterpret_cast<const void*>(qlin_weigh_kernel<__half, 128>)
                        : reinterpret_cast<const void*>(qlin_weigh_kernel<__half, 256>);
}
// A test's: bf16 of width 128.
const void* weigh_fault_fn() { return reinterpret_cast<const void*>(qlin_weigh_kernel<__nv_bfloat16, 128, true>); }

struct WeighDevice {
  std::once_flag once;
  qlin_status ready = QLIN_ERR_CUDA;
  int ctas = 0;
};
WeighDevice g_weigh[64];

qlin_status weigh_setup(int* ctas) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return status_of(e);
  if (dev < 0 || dev >= 64) return QLIN_ERR_CUDA;
  WeighDevice& d = g_weigh[dev];
  std::call_once(d.once, [&d, dev] {
    cudaError_t e = cudaDeviceGetAttribute(&d.ctas, cudaDevAttrMultiProcessorCount, dev);
    auto prepare = [&e](const void* fn) {
      if (e == cudaSuccess) e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, WEIGH_SMEM + 1024);
    };
    for (int dtype : {QLIN_BF16, QLIN_F16})
      for (int width : {64, 128, 256}) prepare(weigh_fn(dtype, width));
    prepare(weigh_fault_fn());
    d.ready = e == cudaSuccess && encode_tiled() && d.ctas > 0 ? QLIN_OK : QLIN_ERR_CUDA;
    if (e != cudaSuccess) (void)cudaGetLastError();
  });
  *ctas = d.ctas;
  return d.ready;
}

qlin_status weigh(const qlin_kv_cache* cache, const qlin_kv_step* step, int Hq, const void* q, int64_t q_stride,
                  const float* stats, float scale, const int32_t* keep, int64_t keep_stride, const int32_t* n_keep,
                  float decay, const float* score, int64_t seq_stride, int64_t head_stride, float* score_out,
                  int32_t* position_out, int64_t out_seq_stride, int64_t out_head_stride, int64_t room,
                  const int32_t* at, void* ws, size_t ws_bytes, unsigned flags, void* stream, int64_t fault_copy) {
  qlin_status st = check_cache(cache);
  if (st != QLIN_OK) return st;
  st = check_step(step, QLIN_MAX_TREE);
  if (st != QLIN_OK) return st;
  if (Hq < 1 || Hq % cache->heads) return QLIN_ERR_INVALID_ARG;
  if ((int64_t)step->T * (Hq / cache->heads) > MAX_ROWS || (int64_t)step->B * cache->heads > (1 << 24))
    return QLIN_ERR_UNSUPPORTED;
  if (flags & ~QLIN_FLAG_PDL) return QLIN_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !std::isfinite(decay) || room < 0) return QLIN_ERR_INVALID_ARG;
  if (room > QLIN_MAX_ROOM) return QLIN_ERR_UNSUPPORTED;
  st = check_status_ws(ws, ws_bytes);
  if (st != QLIN_OK) return st;
  if (step->B == 0 || step->T == 0) return QLIN_OK;
  const int64_t B = step->B, D = cache->width;
  if (!rows_ok(q, q_stride, Hq * D, 2) || !stats || !is_aligned(stats, 8) || !score || !score_out) return QLIN_ERR_INVALID_ARG;
  for (const void* x : {(const void*)keep, (const void*)n_keep, (const void*)at, (const void*)score, (const void*)score_out,
                        (const void*)position_out})
    if (!is_aligned(x, 4)) return QLIN_ERR_INVALID_ARG;
  if ((keep == nullptr) != (n_keep == nullptr) || (keep && keep_stride < step->T)) return QLIN_ERR_INVALID_ARG;
  if (!scores_ok(B, cache->heads, room, seq_stride, head_stride) ||
      !scores_ok(B, cache->heads, room, out_seq_stride, out_head_stride))
    return QLIN_ERR_INVALID_ARG;
  const int64_t span = scores_span(B, cache->heads, room, seq_stride, head_stride) * 4;
  const int64_t out_span = scores_span(B, cache->heads, room, out_seq_stride, out_head_stride) * 4;
  const bool in_place = score == score_out && seq_stride == out_seq_stride && head_stride == out_head_stride;
  if ((!in_place && rows_overlap(score, span, span, score_out, out_span, out_span, 1)) ||
      rows_overlap(score, span, span, position_out, out_span, out_span, 1) ||
      rows_overlap(score_out, out_span, out_span, position_out, out_span, out_span, 1))
    return QLIN_ERR_INVALID_ARG;
  for (const void* out : {(const void*)score_out, (const void*)position_out}) {  // some CTAs write while others still read
    const int64_t rows = B * step->T, heads = Hq;
    if (rows_overlap(out, out_span, out_span, q, (rows - 1) * q_stride * 2 + heads * D * 2, (rows - 1) * q_stride * 2 + heads * D * 2, 1) ||
        rows_overlap(out, out_span, out_span, stats, rows * heads * 8, rows * heads * 8, 1) ||
        rows_overlap(out, out_span, out_span, at, rows * 4, rows * 4, 1))
      return QLIN_ERR_INVALID_ARG;
  }
  int ctas = 0;
  st = weigh_setup(&ctas);
  if (st != QLIN_OK) return st;
  WeighParams p = {};
  p.box = cache->page_size < TILE ? cache->page_size : TILE;
  if (!encode(encode_tiled(), &p.map_k, cache, cache->k, p.box)) return QLIN_ERR_CUDA;
  while ((1 << p.page_shift) < cache->page_size) p.page_shift++;
  p.cache = *cache;
  p.step = *step;
  p.q = q, p.q_stride = q_stride;
  p.stats = reinterpret_cast<const float2*>(stats);
  p.keep = keep, p.n_keep = n_keep, p.keep_stride = keep_stride, p.at = at;
  p.score = score, p.score_out = score_out, p.position_out = position_out;
  p.seq_stride = seq_stride, p.head_stride = head_stride, p.out_seq_stride = out_seq_stride, p.out_head_stride = out_head_stride;
  p.status = static_cast<uint32_t*>(ws);
  p.scale_log2 = (float)((double)scale * 1.4426950408889634);
  p.decay = decay;
  p.room = (int)room;
  p.group = Hq / cache->heads;
  p.group_inverse = (65536u + (uint32_t)p.group - 1) / (uint32_t)p.group;
  p.Rp = (step->T * p.group + 15) / 16 * 16;
  const int q_bytes = p.Rp * cache->width * 2, fit = (WEIGH_SMEM - q_bytes) / SLOT_BYTES;
  p.slots = fit < MAX_SLOTS ? fit : MAX_SLOTS;
  p.ctas = ctas;
  p.fault_copy = fault_copy;
  void* args[] = {&p};
  return launch_step(fault_copy < 0 ? weigh_fn(cache->dtype, cache->width) : weigh_fault_fn(), dim3((unsigned)ctas, 1, 1),
                     dim3(WEIGH_THREADS, 1, 1), (size_t)q_bytes + (size_t)p.slots * SLOT_BYTES + 1024,
                     static_cast<cudaStream_t>(stream), args, (flags & QLIN_FLAG_PDL) != 0);
}

}  // namespace
}  // namespace qlin

using namespace qlin;

extern "C" {

qlin_status qlin_kv_weigh(const qlin_kv_cache* cache, const qlin_kv_step* step, int Hq, const void* q, int64_t q_stride,
                          const float* stats, float scale, const int32_t* keep, int64_t keep_stride,
                          const int32_t* n_keep, float decay, const float* score, int64_t seq_stride,
                          int64_t head_stride, float* score_out, int32_t* position_out, int64_t out_seq_stride,
                          int64_t out_head_stride, int64_t room, const int32_t* at, void* ws, size_t ws_bytes,
                          unsigned flags, void* stream) {
  return weigh(cache, step, Hq, q, q_stride, stats, scale, keep, keep_stride, n_keep, decay, score, seq_stride, head_stride,
               score_out, position_out, out_seq_stride, out_head_stride, room, at, ws, ws_bytes, flags, stream, -1);
}

qlin_status qlin_debug_kv_weigh_fault(const qlin_kv_cache* cache, const qlin_kv_step* step, int Hq, const void* q,
                                      int64_t q_stride, const float* stats, float scale, const float* score,
                                      int64_t seq_stride, int64_t head_stride, float* score_out, int64_t room, void* ws,
                                      size_t ws_bytes, int64_t copy, void* stream) {
  const qlin_status st = check_cache(cache);
  if (st != QLIN_OK) return st;
  if (copy < 0) return QLIN_ERR_INVALID_ARG;
  if (cache->dtype != QLIN_BF16 || cache->width != 128) return QLIN_ERR_UNSUPPORTED;
  return weigh(cache, step, Hq, q, q_stride, stats, scale, nullptr, 0, nullptr, 1.f, score, seq_stride, head_stride, score_out,
               nullptr, seq_stride, head_stride, room, nullptr, ws, ws_bytes, 0, stream, copy);
}

}  // extern "C"
