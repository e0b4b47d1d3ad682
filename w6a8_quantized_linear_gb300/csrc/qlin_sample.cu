// qlin_sample: one token per row of logits under temperature, top-k, top-p and
// min-p, from a given uniform number.
//
// No sort: every filter keeps a beginning of the order (logit descending,
// index ascending), so the kept set is a threshold (key, index) and a bound on
// w.  A threshold is found by counting: a histogram over the logits' range
// finds the bin in which the wanted count (top-k) or mass (top-p) is reached,
// and that bin is split again, first in its range of logits, then in its range
// of 32-bit keys, until one key is left.  Weights are integers (42-bit
// fractions), so all sums are exact and independent of their order.
#include <cmath>
#include <mutex>

#include "qlin_ptx.cuh"
#include "qlin_step.h"

namespace qlin {
namespace {

constexpr int SAMPLE_THREADS = 1024;
constexpr int SAMPLE_WARPS = SAMPLE_THREADS / 32;
constexpr int BINS = 1024;               // one per thread in the scans
constexpr int MAX_C = 16;                // CTAs of a row's cluster, at most
constexpr int ONE_BITS = 42;             // weights are multiples of 2^-42; 2^19 of them sum below 2^62
constexpr uint32_t ALL = 0xFFFFFFFFu;

// 2^(i/32) in units of 2^-31, to the nearest
__constant__ uint32_t TABLE[32] = {
    0x80000000u, 0x82CD8699u, 0x85AAC368u, 0x88980E81u, 0x8B95C1E4u, 0x8EA4398Bu, 0x91C3D374u, 0x94F4EFA9u,
    0x9837F052u, 0x9B8D39BAu, 0x9EF53261u, 0xA2704303u, 0xA5FED6AAu, 0xA9A15AB5u, 0xAD583EEAu, 0xB123F582u,
    0xB504F334u, 0xB8FBAF47u, 0xBD08A39Fu, 0xC12C4CCAu, 0xC5672A11u, 0xC9B9BD86u, 0xCE248C15u, 0xD2A81D92u,
    0xD744FCCBu, 0xDBFBB798u, 0xE0CCDEECu, 0xE5B906E7u, 0xEAC0C6E8u, 0xEFE4B99Cu, 0xF5257D15u, 0xFA83B2DBu,
};

struct SampleParams {
  const void* logits;
  int64_t ld;
  const float *u, *temperature, *top_p, *min_p;
  const int32_t* top_k;
  int32_t* token;
  float* prob;
  int V, slice;  // tokens of the row, of one CTA (a multiple of 32)
};

struct Bin {  // of the whole row, in every CTA
  unsigned long long mass;
  uint32_t count, kmin, kmax, pad;
};
struct Round {  // what the CTAs of a row tell each other outside the histograms
  float mx, mn;
  uint32_t nan, first;
  unsigned long long sum;
};

struct SampleShared {
  uint32_t lo[BINS], hi[BINS], count[BINS], kmin[BINS], kmax[BINS];  // this CTA's histogram
  Bin bins[BINS];
  Round peer[3][MAX_C];
  unsigned long long warp_sum[SAMPLE_WARPS];
  uint32_t warp_a[SAMPLE_WARPS];
  float warp_f[SAMPLE_WARPS], warp_g[SAMPLE_WARPS];
  uint32_t table[32];  // 2^(i/32) in [2^31, 2^32)
  int pick;
  unsigned long long before;
  uint32_t tie;
};

__device__ __forceinline__ uint32_t key_of(float x) {  // larger logit, larger key (no -0 among the logits)
  const uint32_t b = __float_as_uint(x);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// exp((x - max) / T) as a multiple of 2^-42.  With c = log2(e) / T as a pair
// of floats, y = (x - max) c is formed to about 2^-40, split into integer part
// and a 32-bit fraction f; 2^f is a table of 2^(i/32) times the series of
// e^z, z < ln(2)/32 (table and short series: Tang, "Table-driven
// implementation of the exponential function", 1989), its first-order term in
// integers and the rest, below 2^-12, in fp32.
__device__ __forceinline__ unsigned long long weight_of(float x, float mx, float ch, float cl, const uint32_t* table) {
  const float d = x - mx;
  if (!(d < 0.f)) return d == 0.f ? 1ull << ONE_BITS : 0;  // the largest; NaN cannot come here
  const float t = d - x;
  const float e = (x - (d - t)) + (-mx - t);  // d + e = x - mx exactly
  const float yh = d * ch;
  if (!(yh > -(ONE_BITS + 2.f))) return 0;  // below half a unit (-inf too)
  const float yl = fmaf(d, ch, -yh) + fmaf(d, cl, e * ch);
  const long long fix = __float2ll_rn(yh * 4294967296.f) + __float2int_rn(yl * 4294967296.f);
  if (fix >= 0) return 1ull << ONE_BITS;  // yh = 0 and a correction that rounds to it
  const uint32_t f = (uint32_t)fix;
  const int shift = -(int)(fix >> 32);  // >= 1
  const uint32_t z = __umulhi(f << 5, 0xB17217F8u);  // (f mod 1/32) ln 2, in units of 2^-37
  const float zf = (float)z * 0x1p-37f;
  const uint32_t em1 = z + (uint32_t)(zf * zf * fmaf(zf, fmaf(zf, 1.f / 24, 1.f / 6), 0.5f) * 0x1p37f);  // e^z - 1
  const uint32_t base = table[f >> 27];
  const uint32_t m = base + (__umulhi(base, em1) >> 5);  // 2^f in units of 2^-31
  return shift > ONE_BITS + 1 ? 0 : ((((unsigned long long)m << (ONE_BITS - 31 + 1)) >> shift) + 1) >> 1;
}

// Which part of the order survives: keys above `key`, and equal ones up to
// `index` of this CTA's slice.
struct Kept {
  uint32_t key;
  int index;
  __device__ __forceinline__ bool has(uint32_t k, int i) const { return k > key || (k == key && i <= index); }
};

struct Row {
  const float* x;  // this CTA's slice
  int n, w0, w1;   // its tokens, this warp's part of them
  float mx, ch, cl, to_bin;
  uint32_t rank, C;
  SampleShared* s;
};

template <typename T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(ALL, v, o);
  return v;
}

__device__ __forceinline__ void row_sync(const Row& r) {
  if (r.C == 1) {
    __syncthreads();
  } else {
    cluster_arrive();
    cluster_wait();
  }
}

template <typename T>
__device__ __forceinline__ void to_peer(const void* local, uint32_t rank, T v);
template <>
__device__ __forceinline__ void to_peer(const void* local, uint32_t rank, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(dsmem_addr(local, rank)), "r"(v) : "memory");
}
template <>
__device__ __forceinline__ void to_peer(const void* local, uint32_t rank, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(dsmem_addr(local, rank)), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t from_peer(const uint32_t* local, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(dsmem_addr(local, rank)) : "memory");
  return v;
}

__device__ __forceinline__ int bin0(const Row& r, float x) {  // of the row's range of logits
  return min(BINS - 1, (int)((r.mx - x) * r.to_bin));
}
__device__ __forceinline__ int bin1(const Row& r, float x, int b0) {  // of the range of one such bin
  return max(0, min(BINS - 1, (int)(((r.mx - x) * r.to_bin - (float)b0) * (float)BINS)));
}

// The sum over this CTA's threads of v before this thread (exclusive), and
// the total.
__device__ __forceinline__ unsigned long long block_scan(unsigned long long v, unsigned long long* total,
                                                         SampleShared* s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned long long inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long a = __shfl_up_sync(ALL, inc, o);
    if (lane >= o) inc += a;
  }
  __syncthreads();  // the previous scan's sums have been read
  if (lane == 31) s->warp_sum[warp] = inc;
  __syncthreads();
  unsigned long long w = s->warp_sum[lane], winc = w;  // 32 warps, one per lane
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long a = __shfl_up_sync(ALL, winc, o);
    if (lane >= o) winc += a;
  }
  *total = __shfl_sync(ALL, winc, 31);
  return __shfl_sync(ALL, winc - w, warp) + inc - v;
}

// The slice's index of the quota-th token (from 1) with this key among those up
// to `bound`; -1 for none.  All threads of the CTA.
__device__ __forceinline__ int index_of(const Row& r, uint32_t key, int bound, uint32_t quota) {
  if (quota == 0) return -1;
  SampleShared* s = r.s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t n = 0;
  for (int i = r.w0 + lane; i < r.w1; i += 32) n += key_of(r.x[i]) == key && i <= bound;
  n = warp_sum(n);
  if (lane == 0) s->warp_a[warp] = n;
  __syncthreads();
  uint32_t before = 0;
  for (int w = 0; w < warp; w++) before += s->warp_a[w];
  if (before < quota && quota <= before + n) {
    uint32_t left = quota - before;
    for (int i0 = r.w0; i0 < r.w1; i0 += 32) {
      const int i = i0 + lane;
      const uint32_t hit = __ballot_sync(ALL, i < r.w1 && key_of(r.x[i]) == key && i <= bound);
      if ((uint32_t)__popc(hit) >= left) {
        if (lane == 0) s->tie = i0 + __fns(hit, 0, left);
        break;
      }
      left -= __popc(hit);
    }
  }
  __syncthreads();
  return (int)s->tie;
}

// The shortest beginning of the survivors' order whose count (by_mass false)
// reaches `want`, or whose mass reaches the share top_p of theirs; `kept` is
// narrowed to it.  All CTAs of the row take part and agree on everything but
// kept.index, which is of each CTA's own slice.
__device__ __forceinline__ void narrow(const Row& r, Kept& kept, bool by_mass, unsigned long long want, float top_p) {
  SampleShared* s = r.s;
  const int lane = threadIdx.x & 31;
  int b0 = 0, level = 0, sh = 0;
  uint32_t kmax = 0, kmin = 0;
  while (true) {
    for (int i = threadIdx.x; i < BINS; i += SAMPLE_THREADS) {
      s->lo[i] = s->hi[i] = s->count[i] = s->kmax[i] = 0;
      s->kmin[i] = ALL;
    }
    __syncthreads();
    for (int i = r.w0 + lane; i < r.w1; i += 32) {
      const float x = r.x[i];
      const uint32_t key = key_of(x);
      if (x == -INFINITY || !kept.has(key, i)) continue;
      int b;
      if (level == 0) {
        b = bin0(r, x);
      } else if (level == 1) {
        if (bin0(r, x) != b0) continue;
        b = bin1(r, x, b0);
      } else {
        if (key < kmin || key > kmax) continue;
        b = (int)((kmax - key) >> sh);
      }
      atomicAdd(&s->count[b], 1u);
      if (by_mass) {
        const unsigned long long w = weight_of(x, r.mx, r.ch, r.cl, s->table);
        const uint32_t wl = (uint32_t)w;
        const uint32_t wh = (uint32_t)(w >> 32) + ((uint32_t)(atomicAdd(&s->lo[b], wl) + wl) < wl ? 1u : 0u);  // the carry
        if (wh) atomicAdd(&s->hi[b], wh);
      }
      if (level) {
        atomicMin(&s->kmin[b], key);
        atomicMax(&s->kmax[b], key);
      }
    }
    row_sync(r);  // every CTA's histogram is complete
    // each CTA joins its share of the bins and gives them to all
    const int share = BINS / r.C;
    for (int i = threadIdx.x; i < share; i += SAMPLE_THREADS) {
      const int b = r.rank * share + i;
      unsigned long long mass = 0;
      uint32_t count = 0, lo = ALL, hi = 0;
      for (uint32_t c = 0; c < r.C; c++) {
        mass += from_peer(&s->lo[b], c) + ((unsigned long long)from_peer(&s->hi[b], c) << 32);
        count += from_peer(&s->count[b], c);
        lo = min(lo, from_peer(&s->kmin[b], c));
        hi = max(hi, from_peer(&s->kmax[b], c));
      }
      for (uint32_t c = 0; c < r.C; c++) {
        to_peer(&s->bins[b].mass, c, mass);
        to_peer(&s->bins[b].count, c, count);
        to_peer(&s->bins[b].kmin, c, lo);
        to_peer(&s->bins[b].kmax, c, hi);
      }
    }
    row_sync(r);
    const Bin mine = s->bins[threadIdx.x];
    unsigned long long total;
    const unsigned long long v = by_mass ? mine.mass : mine.count;
    const unsigned long long before = block_scan(v, &total, s);
    if (level == 0 && by_mass) {
      const double t = ceil((double)top_p * (double)total);
      want = t < 1. ? 1 : (unsigned long long)t;
      if (want > total) want = total;
    }
    if (total < want || total == 0) return;  // all survivors (the same in every CTA)
    if (before < want && want <= before + v) {
      s->pick = threadIdx.x;
      s->before = before;
    }
    __syncthreads();
    const int b = s->pick;
    want -= s->before;
    const Bin hit = s->bins[b];
    if (level == 0) {
      b0 = b;
    } else {
      kmin = hit.kmin;
      kmax = hit.kmax;
      if (kmin == kmax) {  // one key: its first `want` by index
        if (by_mass) {
          const unsigned long long w = hit.mass / hit.count;  // they weigh the same
          want = w ? (want + w - 1) / w : hit.count;
        }
        const int bound = kmax == kept.key ? kept.index : 0x7FFFFFFF;
        kept.key = kmax;
        kept.index = bound;
        if (want < hit.count) {  // the same in every CTA
          unsigned long long ahead = 0;
          for (uint32_t c = 0; c < r.rank; c++) ahead += from_peer(&s->count[b], c);
          const uint32_t own = s->count[b];
          const uint32_t quota = want <= ahead ? 0 : want - ahead >= own ? own : (uint32_t)(want - ahead);
          if (quota < own) kept.index = index_of(r, kmax, bound, quota);
          row_sync(r);  // the counts have been read
        }
        return;
      }
      sh = 0;
      while (((kmax - kmin) >> sh) >= (uint32_t)BINS) sh++;
    }
    level++;
    __syncthreads();  // pick and bins have been read
  }
}

__device__ __forceinline__ float load_logit(const float* p) { return __ldcs(p) + 0.f; }  // -0 becomes 0
__device__ __forceinline__ float load_logit(const __nv_bfloat16* p) { return __bfloat162float(*p) + 0.f; }

template <typename T>
__global__ void __launch_bounds__(SAMPLE_THREADS) qlin_sample_kernel(const __grid_constant__ SampleParams p, int C) {
  extern __shared__ __align__(16) uint8_t raw[];
  SampleShared* s = reinterpret_cast<SampleShared*>(raw);
  float* x = reinterpret_cast<float*>(raw + sizeof(SampleShared));
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Row r;
  r.x = x;
  r.s = s;
  r.C = C;
  r.rank = C == 1 ? 0 : cluster_ctarank();
  const int row = blockIdx.x / C;
  const int64_t first = (int64_t)r.rank * p.slice;
  r.n = (int)max((int64_t)0, min((int64_t)p.slice, p.V - first));
  const int part = (r.n + 32 * SAMPLE_WARPS - 1) / (32 * SAMPLE_WARPS) * 32;  // contiguous tokens of one warp
  r.w0 = min(r.n, warp * part);
  r.w1 = min(r.n, r.w0 + part);
  if (C > 1) cluster_arrive_relaxed();
  if (threadIdx.x < 32) s->table[threadIdx.x] = TABLE[threadIdx.x];
  pdl_wait();
  pdl_launch_dependents();
  const T* src = static_cast<const T*>(p.logits) + row * p.ld + first;
  float mx = -INFINITY, mn = INFINITY;
  uint32_t nan = 0;
  for (int i = r.w0 + lane; i < r.w1; i += 32) {
    const float v = load_logit(src + i);
    x[i] = v;
    nan |= v != v;
    mx = fmaxf(mx, v);
    if (v > -INFINITY) mn = fminf(mn, v);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    mx = fmaxf(mx, __shfl_xor_sync(ALL, mx, o));
    mn = fminf(mn, __shfl_xor_sync(ALL, mn, o));
    nan |= __shfl_xor_sync(ALL, nan, o);
  }
  if (lane == 0) s->warp_f[warp] = mx, s->warp_g[warp] = mn, s->warp_a[warp] = nan;
  __syncthreads();
  mx = s->warp_f[lane], mn = s->warp_g[lane], nan = s->warp_a[lane];
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    mx = fmaxf(mx, __shfl_xor_sync(ALL, mx, o));
    mn = fminf(mn, __shfl_xor_sync(ALL, mn, o));
    nan |= __shfl_xor_sync(ALL, nan, o);
  }
  if (C > 1) {
    cluster_wait();  // every CTA of the row has started
    if (threadIdx.x < C) {
      to_peer(&s->peer[0][r.rank].mx, threadIdx.x, __float_as_uint(mx));
      to_peer(&s->peer[0][r.rank].mn, threadIdx.x, __float_as_uint(mn));
      to_peer(&s->peer[0][r.rank].nan, threadIdx.x, nan);
    }
    row_sync(r);
    for (int c = 0; c < C; c++) {
      mx = fmaxf(mx, s->peer[0][c].mx);
      mn = fminf(mn, s->peer[0][c].mn);
      nan |= s->peer[0][c].nan;
    }
  }
  if (nan || mx == -INFINITY) {  // no token
    if (r.rank == 0 && threadIdx.x == 0) {
      p.token[row] = -1;
      if (p.prob) p.prob[row] = 0.f;
    }
    return;
  }
  const float temperature = p.temperature ? p.temperature[row] : 1.f;
  if (!(temperature > 0.f)) {
    uint32_t at = ALL;
    for (int i = r.w0 + lane; i < r.w1; i += 32)
      if (x[i] == mx) at = min(at, (uint32_t)(first + i));
    at = __reduce_min_sync(ALL, at);
    __syncthreads();  // warp_a has been read
    if (lane == 0) s->warp_a[warp] = at;
    __syncthreads();
    at = __reduce_min_sync(ALL, s->warp_a[lane]);
    if (C > 1) {
      if (threadIdx.x < C) to_peer(&s->peer[1][r.rank].first, threadIdx.x, at);
      row_sync(r);
      for (int c = 0; c < C; c++) at = min(at, s->peer[1][c].first);
    }
    if (r.rank == 0 && threadIdx.x == 0) {
      p.token[row] = (int32_t)at;
      if (p.prob) p.prob[row] = 1.f;
    }
    return;
  }
  if (mx == INFINITY) {  // the infinite ones are left, alike
    for (int i = r.w0 + lane; i < r.w1; i += 32) x[i] = x[i] == INFINITY ? 0.f : -INFINITY;
    __syncwarp();
    mx = mn = 0.f;
  }
  r.mx = mx;
  const double c = 1.4426950408889634 / (double)temperature;
  r.ch = (float)c;
  r.cl = (float)(c - (double)r.ch);
  r.to_bin = mx - mn > 0.f ? (float)(BINS - 1) / (mx - mn) : 0.f;

  Kept kept = {0u, 0x7FFFFFFF};
  const int top_k = p.top_k ? p.top_k[row] : 0;
  if (top_k > 0 && top_k < p.V) narrow(r, kept, false, (unsigned long long)top_k, 0.f);
  const float top_p = p.top_p ? p.top_p[row] : 1.f;
  if (top_p < 1.f) narrow(r, kept, true, 0, fmaxf(top_p, 0.f));
  const float min_p = p.min_p ? p.min_p[row] : 0.f;
  unsigned long long least = 1;
  if (min_p > 0.f) least = max(1ull, (unsigned long long)ceil((double)fminf(min_p, 1.f) * (double)(1ull << ONE_BITS)));

  // the kept mass of each warp's tokens, of the CTAs, of the row
  unsigned long long mine = 0;
  for (int i = r.w0 + lane; i < r.w1; i += 32) {
    const float v = x[i];
    if (!kept.has(key_of(v), i)) continue;
    const unsigned long long w = weight_of(v, r.mx, r.ch, r.cl, s->table);
    if (w >= least) mine += w;
  }
  mine = warp_sum(mine);
  __syncthreads();  // warp_sum has been read
  if (lane == 0) s->warp_sum[warp] = mine;
  __syncthreads();
  const unsigned long long theirs = s->warp_sum[lane];
  const unsigned long long cta = warp_sum(theirs);
  unsigned long long before = warp_sum(lane < warp ? theirs : 0ull);
  unsigned long long total = cta;
  if (C > 1) {
    if (threadIdx.x < C) to_peer(&s->peer[2][r.rank].sum, threadIdx.x, cta);
    row_sync(r);
    total = 0;
    for (int c2 = 0; c2 < C; c2++) {
      const unsigned long long v = s->peer[2][c2].sum;
      if (c2 < (int)r.rank) before += v;
      total += v;
    }
  }
  const float u = p.u[row];
  unsigned long long target = u > 0.f ? (unsigned long long)((double)fminf(u, 1.f) * (double)total) + 1 : 1;
  if (target > total) target = total;
  if (!(before < target && target <= before + mine)) return;
  for (int i0 = r.w0; i0 < r.w1; i0 += 32) {
    const int i = i0 + lane;
    unsigned long long w = 0;
    if (i < r.w1 && kept.has(key_of(x[i]), i)) {
      w = weight_of(x[i], r.mx, r.ch, r.cl, s->table);
      if (w < least) w = 0;
    }
    unsigned long long inc = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long a = __shfl_up_sync(ALL, inc, o);
      if (lane >= o) inc += a;
    }
    if (before + inc >= target && before + inc - w < target) {
      p.token[row] = (int32_t)(first + i);
      if (p.prob) p.prob[row] = (float)((double)w / (double)total);
    }
    before += __shfl_sync(ALL, inc, 31);
    if (before >= target) return;
  }
}

const void* sample_fn(int dtype) {
  return dtype == QLIN_F32 ? reinterpret_cast<const void*>(qlin_sample_kernel<float>)
                           : reinterpret_cast<const void*>(qlin_sample_kernel<__nv_bfloat16>);
}

std::once_flag g_sample_once[64];
qlin_status g_sample_ready[64];

// the kernels' attributes, once per device
qlin_status sample_setup() {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return status_of(e);
  if (dev < 0 || dev >= 64) return QLIN_ERR_CUDA;
  std::call_once(g_sample_once[dev], [dev] {
    for (int dtype : {QLIN_F32, QLIN_BF16}) {
      cudaError_t e = cudaFuncSetAttribute(sample_fn(dtype), cudaFuncAttributeMaxDynamicSharedMemorySize, 220 * 1024);
      if (e == cudaSuccess) e = cudaFuncSetAttribute(sample_fn(dtype), cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      g_sample_ready[dev] = status_of(e);
      if (e != cudaSuccess) return;
    }
  });
  return g_sample_ready[dev];
}

}  // namespace
}  // namespace qlin

using namespace qlin;

extern "C" qlin_status qlin_sample(int M, int64_t V, int dtype, const void* logits, int64_t ld, const float* u,
                                   const float* temperature, const int32_t* top_k, const float* top_p,
                                   const float* min_p, int32_t* token, float* prob, unsigned flags, void* stream) {
  if (M < 0 || V < 1 || (dtype != QLIN_F32 && dtype != QLIN_BF16)) return QLIN_ERR_INVALID_ARG;
  if (V > QLIN_SAMPLE_MAX_V || M > (1 << 24)) return QLIN_ERR_UNSUPPORTED;
  if (flags & ~QLIN_FLAG_PDL) return QLIN_ERR_INVALID_ARG;
  if (M == 0) return QLIN_OK;
  if (!logits || !is_aligned(logits, dtype == QLIN_F32 ? 4 : 2) || ld < V || !u || !token) return QLIN_ERR_INVALID_ARG;
  for (const void* a : {(const void*)u, (const void*)temperature, (const void*)top_k, (const void*)top_p,
                        (const void*)min_p, (const void*)token, (const void*)prob})
    if (!is_aligned(a, 4)) return QLIN_ERR_INVALID_ARG;
  qlin_status st = sample_setup();
  if (st != QLIN_OK) return st;
  int C = 1;
  while (C < 8 && V > (int64_t)C * 4096) C *= 2;
  if (V > 8 * 32768) C = 16;
  SampleParams p = {logits, ld, u, temperature, top_p, min_p, top_k, token, prob, (int)V,
                    (int)(((V + C - 1) / C + 31) / 32 * 32)};
  void* args[] = {&p, &C};
  return launch_step(sample_fn(dtype), dim3((unsigned)(M * C), 1, 1), dim3(SAMPLE_THREADS, 1, 1),
                     sizeof(SampleShared) + (size_t)p.slice * 4, static_cast<cudaStream_t>(stream), args,
                     (flags & QLIN_FLAG_PDL) != 0, C);
}
