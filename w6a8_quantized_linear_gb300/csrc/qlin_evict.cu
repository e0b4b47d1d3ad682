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

constexpr int SELECT_THREADS = 512, SELECT_WARPS = SELECT_THREADS / 32;
constexpr int BINS = 2048;            // of one pass over 11 bits of the keys
constexpr int MAX_CLUSTER = 16;
constexpr int MAX_STAGED = 40960;     // keys of a block in shared memory at most; those behind are formed again
constexpr int MOVE_THREADS = 256;

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
  int cluster, staged;
  int blocks;  // of the second launch, per item
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
  __align__(16) uint4 sums;               // kept for sure and equals, before and behind the border
  uint4 all[MAX_CLUSTER];
  uint64_t warp[SELECT_WARPS];
  uint32_t bin, above, in_bin;
};

// Exclusive sums over the block of two counts in one word; *all: the whole sum.
__device__ __forceinline__ uint64_t block_scan(uint64_t v, SelectShared* s, uint64_t* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t a = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc += a;
  }
  if (lane == 31) s->warp[warp] = inc;
  __syncthreads();
  uint64_t before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < SELECT_WARPS; w++) {
    if (w < warp) before += s->warp[w];
    sum += s->warp[w];
  }
  __syncthreads();
  *all = sum;
  return before + inc - v;
}
__device__ __forceinline__ uint64_t two(uint32_t a, uint32_t b) { return (uint64_t)b << 32 | a; }

// One cluster per item, a run of places per block, its keys staged in shared
// memory.  The border is found from the keys' upper bits down, 11 at a time: a
// histogram per block, added into the bins' owners, and read by all.
__global__ void __launch_bounds__(SELECT_THREADS) qlin_evict_select_kernel(const __grid_constant__ EvictParams p) {
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ SelectShared sh;
  SelectShared* s = &sh;
  const int C = p.cluster, tid = threadIdx.x;
  const int rank = C > 1 ? (int)cluster_ctarank() : 0;
  const int item = blockIdx.x / C, b = item / p.cache.heads, h = item % p.cache.heads;
  for (int i = tid; i < 3 * BINS; i += SELECT_THREADS) (&s->total[0][0])[i] = 0;
  pdl_wait();
  pdl_launch_dependents();
  const int len = p.step.len[b];
  const int want = p.n_keep[b];
  const bool lost = len > p.room || (int64_t)len > (int64_t)p.step.max_pages * p.cache.page_size;
  const int n = lost || len < 0 ? 0 : len;
  const int stays = want < 0 ? 0 : want < n ? want : n;
  if (rank == 0 && tid == 0) {
    if (lost) report(p.status, QLIN_ERR_BAD_INDEX);
    p.chosen[item] = make_int2(0, lost ? len : len < 0 ? -1 : stays);
  }
  const int per = (n + C - 1) / C, i0 = min(rank * per, n), count = min(per, n - i0);
  const float* score = p.score + b * p.seq_stride + h * p.head_stride + i0;
  const int32_t* position = p.position ? p.position + b * p.seq_stride + h * p.head_stride + i0 : nullptr;
  // what stays in place goes to the other arrays as it is; the emptied places are overwritten by the second launch
  float* score_out = p.score_out + b * p.out_seq_stride + h * p.out_head_stride + i0;
  int32_t* position_out = p.position_out ? p.position_out + b * p.out_seq_stride + h * p.out_head_stride + i0 : nullptr;
  const bool copy_score = score_out != score, copy_position = position_out && position_out != position;
  const int since = p.since ? p.since[b] : 0x7FFFFFFF;
  auto form = [&](float x, int at) { return key_of(x, at < p.first || (p.since && at >= since)); };
#pragma unroll 4
  for (int i = tid; i < count; i += SELECT_THREADS) {
    const float x = score[i];
    const int at = position ? position[i] : i0 + i;
    if (i < p.staged) keys[i] = form(x, at);
    if (i0 + i < stays) {
      if (copy_score) score_out[i] = x;
      if (copy_position) position_out[i] = at;
    }
  }
  if (stays == n || stays == 0) return;  // nothing moves; the whole cluster leaves
  auto key = [&](int i) { return i < p.staged ? keys[i] : form(score[i], position ? position[i] : i0 + i); };
  if (C > 1) {
    cluster_arrive();
    cluster_wait();
  }

  // ---- the border: keys above `border` stay, and the first `ties` of its equals
  uint32_t prefix = 0, border = 0, ties = (uint32_t)stays;
  const int share = BINS / C;  // bins that a block owns
#pragma unroll 1
  for (int pass = 0; pass < 3; pass++) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
    for (int i = tid; i < BINS; i += SELECT_THREADS) s->hist[i] = 0;
    __syncthreads();
#pragma unroll 4
    for (int i = tid; i < count; i += SELECT_THREADS) {
      const uint32_t k = key(i);
      if (pass == 0 || k >> (shift + bits) == prefix) atomicAdd(&s->hist[k >> shift & (BINS - 1) & ((1u << bits) - 1)], 1u);
    }
    __syncthreads();
    const uint32_t total = smem_u32(s->total[pass]);
    for (int i = tid; i < BINS; i += SELECT_THREADS)
      if (s->hist[i]) {
        const uint32_t at = total + (uint32_t)(i % share) * 4;
        cluster_add(C > 1 ? dsmem_addr_u32(at, (uint32_t)(i / share)) : at, s->hist[i]);
      }
    if (C > 1) {
      cluster_arrive();
      cluster_wait();
    } else {
      __syncthreads();
    }
    // a thread's four bins, the highest bins first
    const int bin = BINS - 4 - 4 * tid;
    const uint32_t at = total + (uint32_t)(bin % share) * 4;
    const uint4 c = cluster_load4(C > 1 ? dsmem_addr_u32(at, (uint32_t)(bin / share)) : at);
    uint64_t all;
    uint32_t above = (uint32_t)block_scan(c.x + c.y + c.z + c.w, s, &all);
    const uint32_t counts[4] = {c.w, c.z, c.y, c.x};
#pragma unroll
    for (int e = 0; e < 4; e++) {
      if (above < ties && ties <= above + counts[e]) {
        s->bin = (uint32_t)(bin + 3 - e);
        s->above = above;
        s->in_bin = counts[e];
      }
      above += counts[e];
    }
    __syncthreads();
    prefix = prefix << bits | s->bin;
    ties -= s->above;
    border = prefix << shift;
    if (s->in_bin == ties) {  // the whole bin stays: the border lies below it, and no equals are left to choose from
      border--;               // (never 0: with the bin of key 0 everything would stay)
      ties = 0;
      break;
    }
    __syncthreads();
  }

  // ---- who stays: each thread a run of places in order
  const int run = ((per + SELECT_THREADS - 1) / SELECT_THREADS) | 1;  // odd: no bank twice
  const int from = min(tid * run, count), to = min(from + run, count);
  uint32_t sure_low = 0, sure_high = 0, equal_low = 0, equal_high = 0;
  for (int i = from; i < to; i++) {
    const uint32_t k = key(i);
    const bool low = i0 + i < stays;
    if (k > border) (low ? sure_low : sure_high)++;
    if (k == border) (low ? equal_low : equal_high)++;
  }
  uint64_t sums_low, sums_high;
  const uint64_t before_low = block_scan(two(sure_low, equal_low), s, &sums_low);
  const uint64_t before_high = block_scan(two(sure_high, equal_high), s, &sums_high);
  uint32_t equals_before = (uint32_t)(before_low >> 32) + (uint32_t)(before_high >> 32);  // in this block, in order
  if (tid == 0) s->sums = make_uint4((uint32_t)sums_low, (uint32_t)(sums_low >> 32), (uint32_t)sums_high, (uint32_t)(sums_high >> 32));
  if (C > 1) {
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  if (tid < C) s->all[tid] = cluster_load4(C > 1 ? dsmem_addr(&s->sums, tid) : smem_u32(&s->sums));
  if (C > 1) cluster_arrive();  // no block leaves before its sums have been read
  __syncthreads();
  uint32_t left = ties, mine = 0, holes = 0, movers = 0;  // equals still to be taken; before this block
  for (int r = 0; r < C; r++) {
    const uint4 a = s->all[r];
    const uint32_t low = min(left, a.y), high = min(left - low, a.w);
    const int first = min(r * per, n), end = min(first + per, n);
    const uint32_t size_low = (uint32_t)max(0, min(end, stays) - first);
    if (r == rank) mine = left;
    if (r < rank) holes += size_low - a.x - low, movers += a.z + high;
    left -= low + high;
  }
  auto kept = [&](int i, uint32_t& equals) {
    const uint32_t k = key(i);
    return k > border || (k == border && equals++ < mine);
  };
  uint32_t my_holes = 0, my_movers = 0, equals = equals_before;
  for (int i = from; i < to; i++) {
    const bool stay = kept(i, equals);
    if (i0 + i < stays)
      my_holes += !stay;
    else
      my_movers += stay;
  }
  uint64_t listed;
  const uint64_t before = block_scan(two(my_holes, my_movers), s, &listed);
  int32_t* hole = p.lists + (int64_t)item * 2 * p.half + holes + (uint32_t)before;
  int32_t* mover = p.lists + ((int64_t)item * 2 + 1) * p.half + movers + (uint32_t)(before >> 32);
  equals = equals_before;
  for (int i = from; i < to; i++) {
    const bool stay = kept(i, equals);
    if (i0 + i < stays) {
      if (!stay) *hole++ = i0 + i;
    } else if (stay) {
      *mover++ = i0 + i;
    }
  }
  if (rank == C - 1 && tid == 0) p.chosen[item] = make_int2((int)(movers + (uint32_t)(listed >> 32)), stays);
  if (C > 1) cluster_wait();
}

// A row of keys or values per group of width / 8 threads, 16 bytes each, four
// rows on their way per group.
__global__ void __launch_bounds__(MOVE_THREADS) qlin_evict_move_kernel(const __grid_constant__ EvictParams p) {
  const int item = blockIdx.x / p.blocks, part = blockIdx.x % p.blocks;
  const int b = item / p.cache.heads, h = item % p.cache.heads;
  pdl_wait();
  pdl_launch_dependents();
  const int2 chosen = p.chosen[item];
  const int32_t* holes = p.lists + (int64_t)item * 2 * p.half;
  const int32_t* movers = holes + p.half;
  if (h == 0 && part == 0 && threadIdx.x == 0 && p.len_out && chosen.y >= 0) p.len_out[b] = chosen.y;
  const int lanes = p.cache.width / 8, groups = MOVE_THREADS / lanes * p.blocks;
  const int column = threadIdx.x % lanes * 8;
  constexpr int AHEAD = 4;
  const int64_t head = h * p.cache.head_stride + column;
  for (int u0 = part * (MOVE_THREADS / lanes) + threadIdx.x / lanes; u0 < 2 * chosen.x; u0 += AHEAD * groups) {
    uint4 x[AHEAD];
    int64_t to[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; k++) {
      const int u = u0 + k * groups;
      to[k] = -1;
      if (u >= 2 * chosen.x) continue;
      const int64_t from = token_offset(p.cache, p.step, b, movers[u >> 1]);
      to[k] = token_offset(p.cache, p.step, b, holes[u >> 1]);
      if (from < 0 || to[k] < 0) {
        to[k] = -1;
        report(p.status, QLIN_ERR_BAD_INDEX);
        continue;
      }
      x[k] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(u & 1 ? p.cache.v : p.cache.k) + from + head);
    }
#pragma unroll
    for (int k = 0; k < AHEAD; k++)
      if (to[k] >= 0)
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>((u0 + k * groups) & 1 ? p.cache.v : p.cache.k) + to[k] + head) = x[k];
  }
  const int64_t in = b * p.seq_stride + h * p.head_stride, out = b * p.out_seq_stride + h * p.out_head_stride;
  for (int i = part * MOVE_THREADS + threadIdx.x; i < chosen.x; i += MOVE_THREADS * p.blocks) {
    const int from = movers[i], to = holes[i];
    p.score_out[out + to] = p.score[in + from];
    if (p.position_out) p.position_out[out + to] = p.position ? p.position[in + from] : from;
  }
}

struct EvictDevice {
  std::once_flag once;
  qlin_status ready = QLIN_ERR_CUDA;
  int most = 8;  // CTAs of a cluster
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
    const void* fn = reinterpret_cast<const void*>(qlin_evict_select_kernel);
    cudaError_t e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, MAX_STAGED * 4);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(MAX_CLUSTER, 1, 1);
    cfg.blockDim = dim3(SELECT_THREADS, 1, 1);
    cfg.dynamicSmemBytes = MAX_STAGED * 4;
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
    if (n > 0) d.most = MAX_CLUSTER;
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
  p.cluster = 1;
  while (p.cluster < d->most && p.cluster * 2048 < most && 2 * p.cluster * items <= 2 * d->sms) p.cluster *= 2;
  int64_t staged = (most + p.cluster - 1) / p.cluster;
  p.staged = (int)(staged < MAX_STAGED ? staged : MAX_STAGED);
  int64_t blocks = (4 * d->sms + items - 1) / items, useful = (most * cache->width / 8) / (MOVE_THREADS * 4) + 1;
  p.blocks = (int)(blocks < useful ? blocks : useful);
  void* args[] = {&p};
  st = launch_step(reinterpret_cast<const void*>(qlin_evict_select_kernel), dim3((unsigned)(items * p.cluster), 1, 1),
                   dim3(SELECT_THREADS, 1, 1), (size_t)p.staged * 4, static_cast<cudaStream_t>(stream), args,
                   (flags & QLIN_FLAG_PDL) != 0, p.cluster);
  if (st != QLIN_OK) return st;
  return launch_step(reinterpret_cast<const void*>(qlin_evict_move_kernel), dim3((unsigned)(items * p.blocks), 1, 1),
                     dim3(MOVE_THREADS, 1, 1), 0, static_cast<cudaStream_t>(stream), args, true);
}

}  // extern "C"
