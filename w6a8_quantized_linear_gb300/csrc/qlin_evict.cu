// qlin_kv_evict: the tokens of least accumulated weight leave the cache, head by
// head.
//
// Two launches.  The first chooses: per (sequence, cache head) item the least
// kept key and how many of its equals stay, and lists the places that empty
// before the border and the kept tokens behind it, both in order.  The second
// moves the i-th of these into the i-th of those.  What is read (places from the
// border on) is never written and what is written never read, so moving needs no
// order, and a token that stays where it is costs nothing.
#include <mutex>

#include "qlin_ptx.cuh"
#include "qlin_step.h"

namespace qlin {
namespace {

constexpr int BINS = 2048;            // of one pass over 11 bits of the keys
constexpr int MAX_CLUSTER = 16;
constexpr int MOVE_THREADS = 256, MOVE_WARPS = MOVE_THREADS / 32;
constexpr int MOVE_ITEMS = 1024;      // items whose moves are shared out evenly among their blocks
constexpr uint32_t ALL = 0xFFFFFFFFu;

struct EvictParams {
  qlin_kv_cache cache;
  qlin_kv_step step;
  const float* score;
  const int32_t* position;
  float* score_out;
  int32_t* position_out;
  int64_t seq_stride, head_stride, out_seq_stride, out_head_stride;
  const int32_t *n_keep, *since;
  int32_t* len_out;
  uint32_t* status;
  int2* chosen;    // per item: tokens that move, tokens that are left
  int32_t* lists;  // per item: the emptied places, then the tokens that move there, `half` each
  int64_t half;
  int room, first;
  int cluster, items;
};

// Larger is kept: the scores' order, equal ones by index, NaN below all, what
// is safe by its position above all.
__device__ __forceinline__ uint32_t key_of(float score, bool safe) {
  if (safe) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(score + 0.f);  // one zero
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0;
  return u >> 31 ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ void cluster_add(uint32_t addr, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void cluster_load(uint32_t addr, uint32_t (&v)[2]) {
  asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void cluster_load(uint32_t addr, uint32_t (&v)[4]) {
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint4 cluster_load4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

struct SelectShared {
  uint32_t hist[BINS];
  __align__(16) uint32_t total[3][BINS];  // the cluster's counts of this block's share of the bins
  __align__(16) uint4 sums;               // above the border and equal to it, before place `stays`; the same behind it
  uint4 cta[MAX_CLUSTER], warp[32];
  uint32_t above[32];
  uint32_t bin, over, in_bin;
};

__device__ __forceinline__ uint32_t warp_sum(uint32_t v) { return __reduce_add_sync(ALL, v); }

// Of a run of places in order, with `before` equals in front of it and the counts c
// (above and equal before `stays`, the same behind): those that stay.
__device__ __forceinline__ uint2 staying(uint4 c, uint32_t before, uint32_t ties) {
  const uint32_t left = ties > before ? ties - before : 0, low = min(left, c.y);
  return make_uint2(c.x + low, c.z + min(left - low, c.w));
}

// One cluster per item, a run of places per block, a run of those per warp: lane l
// holds places 32 j + l of it, K of them in registers (K = 0: formed again each
// time), so that ranks come from ballots.  The border is found from the keys' upper
// bits down, 11 at a time: a histogram per block, added into the bins' owners,
// and read by all; where a whole bin stays, what lies below need not be looked at.
// Bound by latency: reads of the length and then of the scores, and per pass (two
// as a rule) the atomics of hot bins, a cluster barrier and reads from the other
// blocks.  17 us of 36 for 131000 tokens of 4 heads (64 blocks), 15 of 49 for 128
// items of up to 9001; keys staged in shared memory and ranks by block-wide sums
// took 33 and 25.
template <int K, int SELECT_THREADS>
__global__ void __launch_bounds__(SELECT_THREADS, K > 16 ? 1 : 1024 / SELECT_THREADS)
    qlin_evict_select_kernel(const __grid_constant__ EvictParams p) {
  constexpr int SELECT_WARPS = SELECT_THREADS / 32, PER = BINS / SELECT_THREADS;  // PER: a thread's bins
  static_assert(PER == 4 || PER == 2, "bins are read 16 or 8 bytes at a time");
  __shared__ SelectShared sh;
  SelectShared* s = &sh;
  const int C = p.cluster, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = C > 1 ? (int)cluster_ctarank() : 0;
  const int item = blockIdx.x / C, b = item / p.cache.heads, h = item % p.cache.heads;
  for (int i = tid; i < 3 * BINS / 4; i += SELECT_THREADS) reinterpret_cast<uint4*>(s->total)[i] = make_uint4(0, 0, 0, 0);
  for (int i = tid; i < BINS / 4; i += SELECT_THREADS) reinterpret_cast<uint4*>(s->hist)[i] = make_uint4(0, 0, 0, 0);
  pdl_wait();
  pdl_launch_dependents();
  const int len = p.step.len[b];
  const int want = p.n_keep[b];
  const int since = p.since ? p.since[b] : 0x7FFFFFFF;
  const bool lost = len > p.room || (int64_t)len > (int64_t)p.step.max_pages * p.cache.page_size;
  const int n = lost || len < 0 ? 0 : len;
  const int stays = want < 0 ? 0 : want < n ? want : n;
  if (rank == 0 && tid == 0) {
    if (lost) report(p.status, QLIN_ERR_BAD_INDEX);
    p.chosen[item] = make_int2(0, lost ? len : len < 0 ? -1 : stays);
  }
  const int per = ((n + C * SELECT_WARPS - 1) / (C * SELECT_WARPS) + 31) / 32 * 32;  // places of a warp
  const int i0 = min((rank * SELECT_WARPS + warp) * per, n), end = min(i0 + per, n), rounds = (end - i0 + 31) / 32;
  const float* score = p.score + b * p.seq_stride + h * p.head_stride;
  const int32_t* position = p.position ? p.position + b * p.seq_stride + h * p.head_stride : nullptr;
  // what stays in place goes to the other arrays as it is; the emptied places are overwritten by the second launch
  float* score_out = p.score_out + b * p.out_seq_stride + h * p.out_head_stride;
  int32_t* position_out = p.position_out ? p.position_out + b * p.out_seq_stride + h * p.out_head_stride : nullptr;
  const bool copy_score = score_out != score, copy_position = position_out && position_out != position;
  auto form = [&](float x, int at) { return key_of(x, at < p.first || (p.since && at >= since)); };

  uint32_t keys[K ? K : 1];
  // of this run: the places before `stays` and those behind it
  const bool copies = (copy_score || copy_position) && i0 < stays;
  auto take = [&](int i, float x, int at) {
    if (copies && i < min(end, stays)) {
      if (copy_score) score_out[i] = x;
      if (copy_position) position_out[i] = at;
    }
  };
  if constexpr (K > 0) {
    float x[K];
#pragma unroll
    for (int j = 0; j < K; j++) {  // all on their way at once
      const int i = i0 + 32 * j + lane;
      x[j] = i < end ? score[i] : 0.f;
      keys[j] = (uint32_t)(position && i < end ? position[i] : i);
    }
#pragma unroll
    for (int j = 0; j < K; j++) {
      const int i = i0 + 32 * j + lane, at = (int)keys[j];
      take(i, x[j], at);
      keys[j] = i < end ? form(x[j], at) : 0;
    }
  } else if (copies) {
#pragma unroll 4
    for (int i = i0 + lane; i < end; i += 32) take(i, score[i], position ? position[i] : i);
  }
  if (stays == n || stays == 0) return;  // nothing moves; the whole cluster leaves
  // f(key, place) for the warp's keys, all lanes at once; behind the end: key 0
  auto each = [&](auto&& f) {
    if constexpr (K > 0) {
#pragma unroll
      for (int j = 0; j < K; j++)
        if (j < rounds) f(keys[j], i0 + 32 * j + lane);
    } else {
#pragma unroll 4
      for (int j = 0; j < rounds; j++) {
        const int i = i0 + 32 * j + lane;
        f(i < end ? form(score[i], position ? position[i] : i) : 0u, i);
      }
    }
  };
  if (C > 1) cluster_arrive();  // the totals are zero
  __syncthreads();

  // ---- the border: keys above it stay, and the first `ties` of its equals
  uint32_t prefix = 0, border = 0, ties = (uint32_t)stays;
  const int share = BINS / C;  // bins that a block owns
#pragma unroll 1
  for (int pass = 0; pass < 3; pass++) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
    if (pass) {
      for (int i = tid; i < BINS / 4; i += SELECT_THREADS) reinterpret_cast<uint4*>(s->hist)[i] = make_uint4(0, 0, 0, 0);
      __syncthreads();
    }
    each([&](uint32_t k, int i) {
      if (i < end && (pass == 0 || k >> (shift + bits) == prefix)) atomicAdd(&s->hist[k >> shift & ((1u << bits) - 1)], 1u);
    });
    if (C > 1 && pass == 0) cluster_wait();
    __syncthreads();
    // a thread's bins, the highest first
    const int bin = BINS - PER * (tid + 1);
    uint32_t counts[PER], mine = 0;
    if (C > 1) {
      const uint32_t at = dsmem_addr_u32(smem_u32(s->total[pass]) + (uint32_t)(bin % share) * 4, (uint32_t)(bin / share));
#pragma unroll
      for (int e = 0; e < PER; e++)
        if (s->hist[bin + e]) cluster_add(at + e * 4, s->hist[bin + e]);
      cluster_arrive();
      cluster_wait();
      cluster_load(at, counts);
    } else {
#pragma unroll
      for (int e = 0; e < PER; e++) counts[e] = s->hist[bin + e];
    }
#pragma unroll
    for (int e = 0; e < PER; e++) mine += counts[e];
    uint32_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t a = __shfl_up_sync(ALL, upto, o);
      if (lane >= o) upto += a;
    }
    if (lane == 31) s->above[warp] = upto;
    __syncthreads();
    uint32_t above = upto - mine + warp_sum(lane < warp ? s->above[lane] : 0);
#pragma unroll
    for (int e = PER - 1; e >= 0; e--) {
      if (above < ties && ties <= above + counts[e]) {
        s->bin = (uint32_t)(bin + e);
        s->over = above;
        s->in_bin = counts[e];
      }
      above += counts[e];
    }
    __syncthreads();
    prefix = prefix << bits | s->bin;
    ties -= s->over;
    border = prefix << shift;
    if (s->in_bin == ties) {  // the whole bin stays: the border lies below it, and no equals are left to choose from
      border--;               // (never 0: with the bin of key 0 everything would stay)
      ties = 0;
      break;
    }
  }

  // ---- who stays
  // (A run lies on one side of place `stays` as a rule: one ballot per 32 keys.)
  const int side = end <= stays ? 0 : i0 >= stays ? 1 : 2;
  uint4 c = make_uint4(0, 0, 0, 0);
  if (side < 2) {
    uint32_t sure = 0, equal = 0;
    each([&](uint32_t k, int i) {
      sure += __popc(__ballot_sync(ALL, k > border));
      if (ties) equal += __popc(__ballot_sync(ALL, i < end && k == border));
    });
    c = side ? make_uint4(0, 0, sure, equal) : make_uint4(sure, equal, 0, 0);
  } else {
    each([&](uint32_t k, int i) {
      const bool low = i < stays;
      c.x += __popc(__ballot_sync(ALL, low && k > border));
      c.z += __popc(__ballot_sync(ALL, !low && k > border));
      if (ties) {
        c.y += __popc(__ballot_sync(ALL, low && k == border));
        c.w += __popc(__ballot_sync(ALL, !low && i < end && k == border));
      }
    });
  }
  if (lane == 0) s->warp[warp] = c;
  __syncthreads();
  if (warp == 0) {
    const uint4 w = lane < SELECT_WARPS ? s->warp[lane] : make_uint4(0, 0, 0, 0);
    const uint4 sum = make_uint4(warp_sum(w.x), warp_sum(w.y), warp_sum(w.z), warp_sum(w.w));
    if (lane == 0) s->sums = sum;
  }
  if (C > 1) {
    cluster_arrive();
    cluster_wait();
    if (tid < C) s->cta[tid] = cluster_load4(dsmem_addr(&s->sums, tid));
    cluster_arrive();  // waited for at the end: no block leaves before its sums have been read
    __syncthreads();
  }
  // this warp's places among all: lane r has block r's counts, lane w then warp w's
  uint32_t equals = 0, holes = 0, movers = 0;
  auto before = [&](uint4 x, int first, int size, bool counted) {  // adds the runs in front, each `size` places from `first` on
    uint32_t inc = x.y + x.w;
    const uint32_t own = inc;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t a = __shfl_up_sync(ALL, inc, o);
      if (lane >= o) inc += a;
    }
    const uint2 stay = staying(x, equals + inc - own, ties);
    const int low = max(0, min(min(first + size, n), stays) - min(first, n));
    holes += warp_sum(counted ? (uint32_t)low - stay.x : 0);
    movers += warp_sum(counted ? stay.y : 0);
    equals += warp_sum(counted ? own : 0);
  };
  if (C > 1) before(lane < C ? s->cta[lane] : make_uint4(0, 0, 0, 0), lane * SELECT_WARPS * per, SELECT_WARPS * per, lane < rank);
  before(lane < SELECT_WARPS ? s->warp[lane] : make_uint4(0, 0, 0, 0), (rank * SELECT_WARPS + lane) * per, per, lane < warp);
  int32_t* hole = p.lists + (int64_t)item * 2 * p.half + holes;
  int32_t* mover = p.lists + ((int64_t)item * 2 + 1) * p.half + movers;
  const uint32_t below = (1u << lane) - 1;
  uint32_t moved = 0;
  auto stays_put = [&](uint32_t k, int i) {
    bool stay = k > border;
    if (ties) {
      const uint32_t equal = __ballot_sync(ALL, i < end && k == border);
      stay |= k == border && equals + __popc(equal & below) < ties;
      equals += __popc(equal);
    }
    return stay;
  };
  if (side < 2) {
    int32_t* list = side ? mover : hole;
    each([&](uint32_t k, int i) {
      const bool stay = stays_put(k, i), listed = i < end && stay == (side == 1);
      const uint32_t m = __ballot_sync(ALL, listed);
      if (listed) list[__popc(m & below)] = i;
      list += __popc(m);
    });
    if (side) moved = (uint32_t)(list - mover);
  } else {
    each([&](uint32_t k, int i) {
      const bool stay = stays_put(k, i);
      const bool empty = i < min(end, stays) && !stay, moves = i < end && i >= stays && stay;
      const uint32_t e = __ballot_sync(ALL, empty), m = __ballot_sync(ALL, moves);
      if (empty) hole[__popc(e & below)] = i;
      if (moves) mover[__popc(m & below)] = i;
      hole += __popc(e);
      mover += __popc(m);
      moved += __popc(m);
    });
  }
  if (rank == C - 1 && warp == SELECT_WARPS - 1 && lane == 0) p.chosen[item] = make_int2((int)(movers + moved), stays);
  if (C > 1) cluster_wait();
}

// All items' moves are laid end to end and shared out evenly among the warps (of
// MOVE_ITEMS items at a time).  A lane finds the rows of one move, then all of
// them copy it: 16 bytes a lane, keys and values of a row of 128 at once, eight
// loads on their way per lane.  Bound by memory: 117 MB (read and written) in 21 us,
// 184 MB in 33 (0.83 of the measured copy); a thread finding its own 16 bytes' place
// issued 113 instructions for them, and was bound by that (38 and 66 us).
template <int D>
__global__ void __launch_bounds__(MOVE_THREADS, 4) qlin_evict_move_kernel(const __grid_constant__ EvictParams p) {
  __shared__ int all_starts[MOVE_ITEMS + 1];
  static_assert(MOVE_WARPS * 33 <= MOVE_ITEMS, "a copy per warp");
  __shared__ int warp_total[MOVE_WARPS];
  __shared__ __align__(16) longlong2 rows[MOVE_WARPS][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int item0 = blockIdx.y * MOVE_ITEMS, items = min(p.items - item0, MOVE_ITEMS);
  int* starts = all_starts;
  pdl_wait();
  pdl_launch_dependents();
  // ---- where each item's moves begin
  if (items <= 32) {  // each warp for itself
    const int2 chosen = lane < items ? p.chosen[item0 + lane] : make_int2(0, -1);
    if (p.len_out && blockIdx.x == 0 && warp == 0 && lane < items && (item0 + lane) % p.cache.heads == 0 && chosen.y >= 0)
      p.len_out[(item0 + lane) / p.cache.heads] = chosen.y;
    int upto = chosen.x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(ALL, upto, o);
      if (lane >= o) upto += a;
    }
    starts += warp * 33;
    starts[lane + 1] = upto;
    if (lane == 0) starts[0] = 0;
    __syncwarp();
  } else {
    constexpr int PER = MOVE_ITEMS / MOVE_THREADS;
    int count[PER], sum = 0;
#pragma unroll
    for (int e = 0; e < PER; e++) {
      const int i = tid * PER + e;
      count[e] = 0;
      if (i >= items) continue;
      const int2 chosen = p.chosen[item0 + i];
      count[e] = chosen.x;
      if (p.len_out && blockIdx.x == 0 && (item0 + i) % p.cache.heads == 0 && chosen.y >= 0)
        p.len_out[(item0 + i) / p.cache.heads] = chosen.y;
      sum += chosen.x;
    }
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(ALL, inc, o);
      if (lane >= o) inc += a;
    }
    if (lane == 31) warp_total[warp] = inc;
    __syncthreads();
    int at = inc - sum + (int)__reduce_add_sync(ALL, lane < warp ? warp_total[lane & (MOVE_WARPS - 1)] : 0);
#pragma unroll
    for (int e = 0; e < PER; e++) {
      const int i = tid * PER + e;
      if (i < items) starts[i] = at;
      at += count[e];
    }
    if (tid == MOVE_THREADS - 1) starts[items] = at;
    __syncthreads();
  }
  const int64_t all = starts[items];
  const int warps = gridDim.x * MOVE_WARPS, w = blockIdx.x * MOVE_WARPS + warp;
  const int first = (int)(all * w / warps), end = (int)(all * (w + 1) / warps);

  constexpr int ROWS = D == 64 ? 2 : 1;        // moves that a warp's lanes cover at once
  constexpr int LOADS = D == 256 ? 2 : 1;      // 16-byte loads of a lane per move
  constexpr int AHEAD = 8 / LOADS;
  constexpr int LANES = 32 / ROWS;             // of a move
  const int sub = lane % LANES;
  uint16_t* const base = static_cast<uint16_t*>(LOADS == 1 && sub >= LANES / 2 ? p.cache.v : p.cache.k) +
                         sub % (D / 8) * 8;
  const int64_t other = static_cast<uint16_t*>(p.cache.v) - static_cast<uint16_t*>(p.cache.k);
  for (int m0 = first; m0 < end; m0 += 32) {
    const int m = m0 + lane;
    longlong2 place = make_longlong2(-1, -1);
    if (m < end) {
      int lo = 0, hi = items;  // the item whose moves hold m: starts[lo] <= m < starts[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        (starts[mid] <= m ? lo : hi) = mid;
      }
      const int item = item0 + lo, b = item / p.cache.heads, h = item % p.cache.heads, i = m - starts[lo];
      const int32_t* list = p.lists + (int64_t)item * 2 * p.half;
      const int to = list[i], from = list[p.half + i];
      place.x = token_offset(p.cache, p.step, b, from);
      place.y = token_offset(p.cache, p.step, b, to);
      const int64_t in = b * p.seq_stride + h * p.head_stride, out = b * p.out_seq_stride + h * p.out_head_stride;
      p.score_out[out + to] = p.score[in + from];
      if (p.position_out) p.position_out[out + to] = p.position ? p.position[in + from] : from;
      if (place.x < 0 || place.y < 0) {
        place.x = -1;
        report(p.status, QLIN_ERR_BAD_INDEX);
      } else {
        place.x += h * p.cache.head_stride, place.y += h * p.cache.head_stride;
      }
    }
    rows[warp][lane] = place;
    __syncwarp();
    const int moves = min(32, end - m0);
#pragma unroll 1
    for (int i0 = 0; i0 < moves; i0 += AHEAD * ROWS) {
      uint4 x[AHEAD][LOADS];
      int64_t to[AHEAD];
#pragma unroll
      for (int u = 0; u < AHEAD; u++) {
        const int i = i0 + u * ROWS + lane / LANES;
        to[u] = -1;
        if (i >= moves) continue;
        const longlong2 r = rows[warp][i];
        if (r.x < 0) continue;
        to[u] = r.y;
        x[u][0] = *reinterpret_cast<const uint4*>(base + r.x);
        if constexpr (LOADS == 2) x[u][1] = *reinterpret_cast<const uint4*>(base + other + r.x);
      }
#pragma unroll
      for (int u = 0; u < AHEAD; u++) {
        if (to[u] < 0) continue;
        *reinterpret_cast<uint4*>(base + to[u]) = x[u][0];
        if constexpr (LOADS == 2) *reinterpret_cast<uint4*>(base + other + to[u]) = x[u][1];
      }
    }
    __syncwarp();
  }
}

// Keys of a lane in registers: as many as the longest sequence may need.
struct Select {
  const void* fn;
  int threads;
};
template <int K, int THREADS>
Select select_of() {
  return {reinterpret_cast<const void*>(qlin_evict_select_kernel<K, THREADS>), THREADS};
}
constexpr int64_t SIZES[4] = {2048, 8192, 16384, 16385};  // of the blocks that make clusters (the last: any more)
int size_of(int64_t places) { return places <= SIZES[0] ? 0 : places <= SIZES[1] ? 1 : places <= SIZES[2] ? 2 : 3; }
Select select_fn(int64_t places, int cluster) {  // places of a block
  if (cluster == 1 && places > 2048 && places <= 16384)
    return places <= 4096 ? select_of<4, 1024>() : places <= 8192 ? select_of<8, 1024>() : select_of<16, 1024>();
  switch (size_of(places)) {
    case 0: return select_of<4, 512>();
    case 1: return select_of<16, 512>();
    case 2: return select_of<32, 512>();
    default: return select_of<0, 512>();
  }
}
const void* move_fn(int width) {
  return width == 64    ? reinterpret_cast<const void*>(qlin_evict_move_kernel<64>)
         : width == 128 ? reinterpret_cast<const void*>(qlin_evict_move_kernel<128>)
                        : reinterpret_cast<const void*>(qlin_evict_move_kernel<256>);
}

struct EvictDevice {
  std::once_flag once;
  qlin_status ready = QLIN_ERR_CUDA;
  int most = 8;     // CTAs of a cluster
  int at_once[4] = {};  // clusters of 16 that find room at the same time, by their blocks' size
  int sms = 0;
};
EvictDevice g_evict[64];

qlin_status evict_setup(EvictDevice** device) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return status_of(e);
  if (dev < 0 || dev >= 64) return QLIN_ERR_CUDA;
  EvictDevice& d = g_evict[dev];
  std::call_once(d.once, [&d, dev] {
    cudaError_t e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
    int clusters = 64;
    for (int size = 0; size < 4; size++) {
      const Select select = select_fn(SIZES[size], MAX_CLUSTER);
      const void* fn = select.fn;
      if (e == cudaSuccess) e = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(MAX_CLUSTER, 1, 1);
      cfg.blockDim = dim3((unsigned)select.threads, 1, 1);
      cudaLaunchAttribute attr;
      attr.id = cudaLaunchAttributeClusterDimension;
      attr.val.clusterDim.x = MAX_CLUSTER;
      attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
      cfg.attrs = &attr;
      cfg.numAttrs = 1;
      int n = 0;
      if (e == cudaSuccess && cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();
        n = 0;
      }
      d.at_once[size] = n;
      if (n < clusters) clusters = n;
    }
    if (clusters > 0) d.most = MAX_CLUSTER;
    d.ready = d.sms > 0 ? status_of(e) : QLIN_ERR_CUDA;
  });
  *device = &d;
  return d.ready;
}

constexpr int64_t aligned256(int64_t n) { return (n + 255) / 256 * 256; }
qlin_status check_items(const qlin_kv_cache* c, int64_t B, int64_t room) {
  if (B < 0 || room < 0) return QLIN_ERR_INVALID_ARG;
  if (room > QLIN_MAX_ROOM || B * c->heads > (1 << 20)) return QLIN_ERR_UNSUPPORTED;
  return QLIN_OK;
}

}  // namespace
}  // namespace qlin

using namespace qlin;

extern "C" {

qlin_status qlin_kv_evict_workspace_bytes(const qlin_kv_cache* cache, int B, int64_t room, size_t* bytes) {
  qlin_status st = check_cache(cache);
  if (st != QLIN_OK) return st;
  st = check_items(cache, B, room);
  if (st != QLIN_OK) return st;
  if (!bytes) return QLIN_ERR_INVALID_ARG;
  const int64_t items = (int64_t)B * cache->heads;
  *bytes = (size_t)(STEP_WS_HEADER + aligned256(items * 8) + items * 2 * (room / 2 + 1) * 4);
  return QLIN_OK;
}

qlin_status qlin_kv_evict(const qlin_kv_cache* cache, const qlin_kv_step* step, const float* score,
                          const int32_t* position, int64_t seq_stride, int64_t head_stride, float* score_out,
                          int32_t* position_out, int64_t out_seq_stride, int64_t out_head_stride, int64_t room,
                          const int32_t* n_keep, int first, const int32_t* since, int32_t* len_out, void* ws,
                          size_t ws_bytes, unsigned flags, void* stream) {
  qlin_status st = check_cache(cache);
  if (st != QLIN_OK) return st;
  st = check_step(step, 0x7FFFFFFF);
  if (st != QLIN_OK) return st;
  size_t need = 0;
  st = qlin_kv_evict_workspace_bytes(cache, step->B, room, &need);
  if (st != QLIN_OK) return st;
  if (flags & ~QLIN_FLAG_PDL) return QLIN_ERR_INVALID_ARG;
  if (first < 0) return QLIN_ERR_INVALID_ARG;
  if (step->B == 0 || step->T == 0) return QLIN_OK;
  if (!score || !score_out || !n_keep) return QLIN_ERR_INVALID_ARG;
  for (const void* x : {(const void*)score, (const void*)position, (const void*)score_out, (const void*)position_out,
                        (const void*)n_keep, (const void*)since, (const void*)len_out})
    if (!is_aligned(x, 4)) return QLIN_ERR_INVALID_ARG;
  if (!scores_ok(step->B, cache->heads, room, seq_stride, head_stride) ||
      !scores_ok(step->B, cache->heads, room, out_seq_stride, out_head_stride))
    return QLIN_ERR_INVALID_ARG;
  // in place, or apart
  const bool same = seq_stride == out_seq_stride && head_stride == out_head_stride;
  const int64_t span = scores_span(step->B, cache->heads, room, seq_stride, head_stride) * 4;
  const int64_t out_span = scores_span(step->B, cache->heads, room, out_seq_stride, out_head_stride) * 4;
  auto clash = [&](const void* in, const void* out) {
    return in && out && !(in == out && same) && rows_overlap(in, span, span, out, out_span, out_span, 1);
  };
  if (clash(score, score_out) || clash(position, position_out) || rows_overlap(score, span, span, position_out, out_span, out_span, 1) ||
      rows_overlap(position, span, span, score_out, out_span, out_span, 1) ||
      rows_overlap(score_out, out_span, out_span, position_out, out_span, out_span, 1))
    return QLIN_ERR_INVALID_ARG;
  if (!ws || !is_aligned(ws, 256)) return QLIN_ERR_INVALID_ARG;
  if (ws_bytes < need) return QLIN_ERR_WORKSPACE;
  EvictDevice* d = nullptr;
  st = evict_setup(&d);
  if (st != QLIN_OK) return st;
  const int64_t items = (int64_t)step->B * cache->heads;
  EvictParams p = {};
  p.cache = *cache;
  p.step = *step;
  p.score = score, p.position = position, p.score_out = score_out, p.position_out = position_out;
  p.seq_stride = seq_stride, p.head_stride = head_stride, p.out_seq_stride = out_seq_stride, p.out_head_stride = out_head_stride;
  p.n_keep = n_keep, p.since = since, p.len_out = len_out;
  p.status = static_cast<uint32_t*>(ws);
  p.chosen = reinterpret_cast<int2*>(static_cast<uint8_t*>(ws) + STEP_WS_HEADER);
  p.lists = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + STEP_WS_HEADER + aligned256(items * 8));
  p.half = room / 2 + 1;
  p.room = (int)room, p.first = first;
  int64_t most = (int64_t)step->max_pages * cache->page_size;  // tokens of a sequence
  most = most < room ? most : room;
  p.items = (int)items;
  p.cluster = 1;
  // One block of 1024 threads per item spares the clusters' barriers (four items of
  // 2094 tokens 8.7 us, against 10.2 in clusters of two; 128 of 4000 24.6 and 27.5,
  // of up to 12000 61.1 and 63.5), but leaves SMs idle where items are few and long
  // (eight of 8000 13.9 us against 13.1).  Clusters of 16 (one item of 93375 tokens
  // 14.4 us, 18.5 with eight) where all find room at once: they are placed within a
  // part of the device (16 items of 60000 41.6 us, 35.2 with eight).  All this goes by
  // what the table and the scores have room for, as lengths are known on the device
  // alone: with eight times the room four heads of 131000 tokens take 57 us, 36 without
  // (their keys are formed again in each pass), 128 items of up to 9001 70 and 48.
  if (most > (2 * items >= d->sms ? 16384 : 4096))
    while (p.cluster < d->most && p.cluster * 2048 < most && 2 * p.cluster * items <= 2 * d->sms &&
           (p.cluster < 8 || items <= d->at_once[size_of((most + MAX_CLUSTER - 1) / MAX_CLUSTER)]))
      p.cluster *= 2;
  const Select select = select_fn((most + p.cluster - 1) / p.cluster, p.cluster);
  void* args[] = {&p};
  st = launch_step(select.fn, dim3((unsigned)(items * p.cluster), 1, 1), dim3((unsigned)select.threads, 1, 1), 0,
                   static_cast<cudaStream_t>(stream), args, (flags & QLIN_FLAG_PDL) != 0, p.cluster);
  if (st != QLIN_OK) return st;
  const int64_t groups = (items + MOVE_ITEMS - 1) / MOVE_ITEMS;
  int64_t blocks = (4 * d->sms + groups - 1) / groups;
  const int64_t useful = items * (most / 2) / (8 * MOVE_WARPS) + 1;  // eight moves a warp
  if (blocks > useful) blocks = useful;
  return launch_step(move_fn(cache->width), dim3((unsigned)blocks, (unsigned)groups, 1), dim3(MOVE_THREADS, 1, 1), 0,
                     static_cast<cudaStream_t>(stream), args, true);
}

}  // extern "C"
