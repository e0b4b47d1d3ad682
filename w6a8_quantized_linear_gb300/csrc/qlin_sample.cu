// qlin_sample: one token per row of logits under temperature, top-k, top-p and
// min-p, from a given uniform number.
//
// No sort: every filter keeps a beginning of the order (logit descending,
// index ascending), so the kept set is a threshold (logit, index) and a bound
// on w.  A threshold is found by counting: a histogram over the logits' range
// finds the bin in which the wanted count (top-k) or mass (top-p) is reached;
// a bin of few tokens is settled by comparing them, one of many is split again
// by its range of 32-bit keys, until one key is left.  Weights are integers
// (42-bit fractions), so all sums are exact and independent of their order.
// (Bitonic sorts of the survivors and of a bin, in place of those steps,
// measured 1.4 us slower on one and eight rows.)
#include <cfloat>
#include <cmath>
#include <mutex>
#include <type_traits>

#include "qlin_ptx.cuh"
#include "qlin_sample_weight.h"
#include "qlin_step.h"

namespace qlin {
namespace {

constexpr int SAMPLE_THREADS = 512;
constexpr int SAMPLE_WARPS = SAMPLE_THREADS / 32;
constexpr int BINS = SAMPLE_THREADS;     // one per thread in the scans
constexpr int GROUPS = BINS / 32;
constexpr int MAX_C = 16;                // CTAs of a row's cluster, at most
constexpr int CHUNK = 128;               // consecutive tokens that a warp takes at once, four per lane
constexpr int FEW = 128;                 // a bin of at most this many tokens is settled by comparing all pairs, four threads each
constexpr int LIST = 2048;               // so many tokens, what top-k may leave, are carried on by one CTA
constexpr int OWN = 64;                  // of them from one warp at most
constexpr uint32_t ALL = 0xFFFFFFFFu;

__constant__ uint32_t TABLE[32] = QLIN_EXP2_TABLE;

struct SampleParams {
  const void* logits;
  int64_t ld;
  const float *u, *temperature, *top_p, *min_p;
  const int32_t* top_k;
  int32_t* token;
  float* prob;
  int V, slice;  // tokens of the row, of one CTA (a multiple of CHUNK)
};

struct Round {  // what the CTAs of a row tell each other outside the histograms
  uint32_t kmx, kmn, nan, top, left, pad;
  unsigned long long sum;
};
struct __align__(16) Candidate {
  uint32_t key, index;  // in the row
  unsigned long long weight;
};

struct SampleShared {
  __align__(16) uint32_t hist[3][BINS];  // this CTA's histogram: counts, masses' low and high words
  unsigned long long mass[MAX_C][32];    // a group of bins, by CTAs
  uint32_t count[MAX_C][32];
  Candidate few[FEW];
  uint32_t reach[MAX_C * SAMPLE_WARPS];  // by warps of the row: the key that so many of its tokens reach
  Round peer[2][MAX_C];
  unsigned long long warp_sum[SAMPLE_WARPS];
  uint32_t warp_a[SAMPLE_WARPS], warp_b[SAMPLE_WARPS], warp_c[SAMPLE_WARPS], warp_d[SAMPLE_WARPS];
  uint32_t table[32];  // 2^(i/32) in [2^31, 2^32)
  int pick;
  uint32_t pick_key, pick_index, pick_count, filled;
  unsigned long long before, pick_mass;
};

__device__ __forceinline__ uint32_t key_of(float x) {  // larger logit, larger key (no -0 among the logits)
  const uint32_t b = __float_as_uint(x);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float logit_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

// ceil or floor of n * f for n below 2^62 and f in [0, 1], exactly: f is a
// 24-bit integer over a power of two.  (fp64 is slow here.)
template <bool CEIL>
__device__ __forceinline__ unsigned long long share_of(unsigned long long n, float f) {
  const uint32_t bits = __float_as_uint(f), e = bits >> 23;
  const unsigned long long m = e ? (bits & 0x7FFFFFu) | 0x800000u : bits & 0x7FFFFFu;
  const int shift = 150 - (int)(e ? e : 1);  // f = m 2^-shift, 23 <= shift <= 149
  unsigned long long lo = n * m, hi = __umul64hi(n, m);
  if (CEIL) {  // 2^shift - 1 more; n m + 2^shift stays below 2^127 unless the result is 0 or 1
    if (shift >= 126) return lo | hi ? 1 : 0;
    const unsigned long long al = shift < 64 ? (1ull << shift) - 1 : ~0ull, ah = shift < 64 ? 0 : (1ull << (shift - 64)) - 1;
    const unsigned long long s = lo + al;
    hi += ah + (s < lo);
    lo = s;
  }
  if (shift >= 128) return 0;
  return shift >= 64 ? hi >> (shift - 64) : (lo >> shift) | (hi << (64 - shift));
}

// a / b to 2^-31 and rounded, for 0 < a <= b: an integer division of the
// numbers' leading 64 and 32 bits (fp64 division would cost a microsecond here)
__device__ __forceinline__ float ratio(unsigned long long a, unsigned long long b) {
  const int za = __clzll(a), zb = __clzll(b);
  const unsigned long long q = (a << za) / ((b << zb) >> 32);  // in [2^31, 2^33]
  return ldexpf((float)q, zb - za - 32);
}

// the largest; NaN if one is
__device__ __forceinline__ float max_of(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}
__device__ __forceinline__ float max_of(const float (&v)[4]) { return max_of(max_of(v[0], v[1]), max_of(v[2], v[3])); }

// Which part of the order survives: logits above x, and equal ones up to
// `index` in the row (a bound that only this CTA's tokens have to agree with).
// Forbidden tokens (-inf) never do.
struct Kept {
  float x;
  int index;
  __device__ __forceinline__ bool has(float v, int i) const { return v > x || (v == x && i <= index); }
};
__device__ __forceinline__ Kept everything() { return {-INFINITY, -1}; }

// The tokens that a CTA works on, filled up with -inf to whole chunks per warp:
// a slice of the row in shared memory (STAGED), or where it is, or (one CTA)
// the survivors of top-k.
template <typename T, int CHUNKS, bool STAGED = true>
struct Row {
  using Four = std::conditional_t<sizeof(T) == 4, float4, uint2>;
  static constexpr int KEY_BITS = 8 * sizeof(T);  // leading bits that tell keys apart
  const T* x;
  // The largest of this lane's four tokens in each of its warp's chunks; not
  // STAGED two in a word, rounded up to bf16.
  std::conditional_t<STAGED, float, uint32_t> top[STAGED ? CHUNKS : CHUNKS / 2];
  int w0, w1;        // this warp's contiguous part
  int first;         // index of the slice's first token
  int tokens;        // those of the row in the slice
  bool wide, inf;    // in memory four tokens at a time; not STAGED: the infinite ones are left, alike
  float mx, mn, to_bin;  // mn: nothing that is left is below it
  Weighing weighing;
  uint32_t rank, C;
  SampleShared* s;
  uint32_t* all;     // [C][BINS]: the CTAs' counts
  unsigned long long* group;  // [C][GROUPS]: the CTAs' masses of 32 bins at a time
  __device__ __forceinline__ unsigned long long weight(float v) const { return weight_of(v, weighing, s->table); }
  __device__ __forceinline__ void part(int tokens) {  // whole chunks, alike for all warps
    const int per = (tokens + CHUNK * SAMPLE_WARPS - 1) / (CHUNK * SAMPLE_WARPS) * CHUNK;
    w0 = (threadIdx.x >> 5) * per;
    w1 = w0 + per;
  }
  // tokens 4 lane .. 4 lane + 3 of the chunk at i of the slice in memory
  __device__ __forceinline__ Four fetch(const T* from, int i) const {
    i += (threadIdx.x & 31) * 4;
    const T* at = from + i;
    if (wide && i + 4 <= tokens) return *reinterpret_cast<const Four*>(at);
    T v[4];
#pragma unroll
    for (int e = 0; e < 4; e++) v[e] = i + e < tokens ? at[e] : T(-INFINITY);
    if constexpr (sizeof(T) == 4) {
      return {v[0], v[1], v[2], v[3]};
    } else {
      auto two = [](T a, T b) { return (uint32_t)__bfloat16_as_ushort(a) | (uint32_t)__bfloat16_as_ushort(b) << 16; };
      return {two(v[0], v[1]), two(v[2], v[3])};
    }
  }
  __device__ __forceinline__ Four load(int i) const {
    if constexpr (STAGED) return *reinterpret_cast<const Four*>(x + i + (threadIdx.x & 31) * 4);
    else return fetch(x, i);
  }
  __device__ __forceinline__ void values(const Four& f, float (&v)[4]) const {
    if constexpr (sizeof(T) == 4) {
      v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
    } else {
      const float2 a = unpack2(f.x, T()), b = unpack2(f.y, T());
      v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
    }
#pragma unroll
    for (int e = 0; e < 4; e++) {
      v[e] += 0.f;  // -0 becomes 0
      if constexpr (!STAGED)
        if (inf) v[e] = v[e] == INFINITY ? 0.f : -INFINITY;
    }
  }
  __device__ __forceinline__ void four(int i, float (&v)[4]) const { values(load(i), v); }
  // f(i, v) for the chunks named by `m`, in order; not STAGED with AHEAD more
  // on their way.
  template <typename F>
  __device__ __forceinline__ void each(uint32_t m, const F& f) const {
    if constexpr (STAGED) {
      for (; m; m &= m - 1) {
        float v[4];
        const int i = w0 + (__ffs(m) - 1) * CHUNK;
        four(i, v);
        f(i, v);
      }
    } else {
      float v[4];
      constexpr int AHEAD = sizeof(T) == 4 ? 2 : 3;
      Four next[AHEAD];
      uint32_t far = m;
#pragma unroll
      for (int a = 0; a < AHEAD; a++, far &= far - 1)
        if (far) next[a] = load(w0 + (__ffs(far) - 1) * CHUNK);
      for (; m; m &= m - 1, far &= far - 1) {
        const Four now = next[0];
#pragma unroll
        for (int a = 0; a + 1 < AHEAD; a++) next[a] = next[a + 1];
        if (far) next[AHEAD - 1] = load(w0 + (__ffs(far) - 1) * CHUNK);
        values(now, v);
        f(w0 + (__ffs(m) - 1) * CHUNK, v);
      }
    }
  }
  __device__ __forceinline__ void set_top(int c, float t) {
    if constexpr (STAGED) {
      top[c] = t;
    } else {
      const uint32_t up = __bfloat16_as_ushort(__float2bfloat16_ru(t));
      top[c / 2] = c & 1 ? (top[c / 2] & 0xFFFFu) | up << 16 : up | 0xFF800000u;
    }
  }
  __device__ __forceinline__ void no_top(int c) {
    if constexpr (STAGED) top[c] = -INFINITY;
    else if (c % 2 == 0) top[c / 2] = 0xFF80FF80u;
  }
  __device__ __forceinline__ void tops() {
#pragma unroll
    for (int c = 0; c < CHUNKS; c++) {
      no_top(c);
      if (w0 + c * CHUNK < w1) {
        float v[4];
        four(w0 + c * CHUNK, v);
        set_top(c, max_of(v));
      }
    }
  }
  // The warp's chunks in which some token reaches `least`, as bits: most
  // passes look for a few tokens and read only these.
  __device__ __forceinline__ uint32_t chunks(float least) const {
    uint32_t m = 0;
#pragma unroll
    for (int c = 0; c < CHUNKS; c++) {
      float t;
      if constexpr (STAGED) t = top[c];
      else t = __uint_as_float(c & 1 ? top[c / 2] & 0xFFFF0000u : top[c / 2] << 16);
      m |= (__any_sync(0xFFFFFFFFu, t >= least) ? 1u : 0u) << c;
    }
    return m & ((2u << ((w1 - w0) / CHUNK - 1)) - 1);
  }
  // Place among the row's BINS equal parts of its logits' range, largest
  // first, whole bins as integers: it falls with x, the same in every use.
  __device__ __forceinline__ float place(float v) const { return fminf((mx - v) * to_bin, (float)(BINS - 1)); }
};

__device__ __forceinline__ uint32_t warp_sum(uint32_t v) { return __reduce_add_sync(ALL, v); }

// of numbers below 2^62, in three parts of 27 bits: three reductions at a time
// instead of ten shuffles, five in a row
__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
  constexpr uint32_t PART = (1u << 27) - 1;
  const uint32_t a = __reduce_add_sync(ALL, (uint32_t)v & PART), b = __reduce_add_sync(ALL, (uint32_t)(v >> 27) & PART),
                 c = __reduce_add_sync(ALL, (uint32_t)(v >> 54));
  return a + ((unsigned long long)b << 27) + ((unsigned long long)c << 54);
}

// of v in this lane and those before it
template <typename T>
__device__ __forceinline__ T warp_scan(T v) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T a = __shfl_up_sync(ALL, v, o);
    if ((threadIdx.x & 31) >= o) v += a;
  }
  return v;
}

template <typename R>
__device__ __forceinline__ void row_sync(const R& r) {
  if (r.C == 1) {
    __syncthreads();
  } else {
    cluster_arrive();
    cluster_wait();
  }
}

__device__ __forceinline__ void to_peer(const void* local, uint32_t rank, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(dsmem_addr(local, rank)), "r"(v) : "memory");
}
__device__ __forceinline__ void to_peer(const void* local, uint32_t rank, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(dsmem_addr(local, rank)), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t from_peer(const uint32_t* local, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(dsmem_addr(local, rank)) : "memory");
  return v;
}

// The sum over this CTA's threads of v before this thread (exclusive), and
// the total.
__device__ __forceinline__ unsigned long long block_scan(unsigned long long v, unsigned long long* total,
                                                         SampleShared* s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned long long inc = warp_scan(v);
  __syncthreads();  // the previous scan's sums have been read
  if (lane == 31) s->warp_sum[warp] = inc;
  __syncthreads();
  const unsigned long long w = lane < SAMPLE_WARPS ? s->warp_sum[lane] : 0;
  *total = warp_sum(w);
  return warp_sum(lane < warp ? w : 0ull) + inc - v;
}

// The row index of the quota-th token (from 1) with this logit among the
// survivors of this CTA; -1 for none.  All threads of the CTA.
template <typename R>
__device__ __forceinline__ int index_of(const R& r, const Kept& kept, float x, uint32_t quota) {
  if (quota == 0) return -1;
  SampleShared* s = r.s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto hits = [&](int i0, const float (&v)[4]) -> uint32_t {  // a bit for each of a lane's four tokens
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 4; e++) m |= (v[e] == x && kept.has(v[e], r.first + i0 + lane * 4 + e) ? 1u : 0u) << e;
    return m;
  };
  uint32_t n = 0;
  const uint32_t chunks = r.chunks(x);
  r.each(chunks, [&](int i, const float (&v)[4]) { n += __popc(hits(i, v)); });
  n = warp_sum(n);
  if (lane == 0) s->warp_a[warp] = n;
  __syncthreads();
  uint32_t before = 0;
  for (int w = 0; w < warp; w++) before += s->warp_a[w];
  if (before < quota && quota <= before + n) {
    for (uint32_t k = chunks; k && before < quota; k &= k - 1) {
      const int i = r.w0 + (__ffs(k) - 1) * CHUNK;
      float v[4];
      r.four(i, v);
      const uint32_t m = hits(i, v), c = __popc(m);
      const uint32_t inc = warp_scan(c);
      if (before + inc >= quota && before + inc - c < quota)
        s->pick_index = (uint32_t)(r.first + i + lane * 4 + __fns(m, 0, quota - (before + inc - c)));
      before += __shfl_sync(ALL, inc, 31);
    }
  }
  __syncthreads();
  return (int)s->pick_index;
}

// This CTA's counts to all CTAs of the row.
template <typename R>
__device__ __forceinline__ void push_counts(const R& r) {
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < r.C * (BINS / 4); i += SAMPLE_THREADS) {
    const uint32_t c = i / (BINS / 4), q = i % (BINS / 4) * 4;
    const uint4 x = *reinterpret_cast<const uint4*>(&r.s->hist[0][q]);
    asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dsmem_addr(r.all + r.rank * BINS + q, c)),
                 "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w)
                 : "memory");
  }
}

// A token of weight w in bin b of this CTA's histogram.
__device__ __forceinline__ void add_mass(SampleShared* s, int b, unsigned long long w) {
  atomicAdd(&s->hist[0][b], 1u);
  const uint32_t wl = (uint32_t)w;
  const uint32_t wh = (uint32_t)(w >> 32) + ((uint32_t)(atomicAdd(&s->hist[1][b], wl) + wl) < wl ? 1u : 0u);  // the carry
  if (wh) atomicAdd(&s->hist[2][b], wh);
}

// The lowest and the highest key whose logits fall into bin b of the row's
// range: 16 lanes try as many keys at once for either.  All warps alike, no
// exchange.  (The tokens' own lowest and highest took a pass and an exchange.)
template <typename R>
__device__ __forceinline__ void keys_of_bin(const R& r, const Kept& kept, int b, uint32_t* kmin, uint32_t* kmax) {
  const int lane = threadIdx.x & 31;
  const bool up = lane < 16;  // the highest: upwards from the survivors' lowest
  const uint32_t lowest = key_of(fmaxf(kept.x, r.mn)), highest = key_of(r.mx), i = lane % 16 + 1;
  uint32_t at = 0, len = highest - lowest;  // `at` steps are not too far; what is sought is at most len further
  while (__any_sync(ALL, len)) {
    const uint32_t step = len / 16 + 1, y = at + min(i * step, len);
    const int bin = (int)r.place(logit_of(up ? lowest + y : highest - y));
    const uint32_t hits = __ballot_sync(ALL, up ? bin >= b : bin <= b);  // a half's come first
    const uint32_t n = __popc(up ? hits & 0xFFFFu : hits >> 16), to = min(n * step, len);
    len = n == 16 ? 0 : min((n + 1) * step, len + 1) - 1 - to;  // a try at `len` may have failed: it is made again
    at += to;
  }
  *kmax = lowest + __shfl_sync(ALL, at, 0);
  *kmin = highest - __shfl_sync(ALL, at, 16);
}

// The shortest beginning of the survivors' order whose count (BY_MASS false)
// reaches `want`, or whose mass reaches the share top_p of theirs; `kept` is
// narrowed to it.  All CTAs of the row take part.  Each level costs one
// exchange: histograms of counts are pushed to every CTA; of masses, three
// times the bytes, only the sums of 32 bins, and each CTA then reads the 32
// bins in which the border lies from the others (all bins joined by shares
// took a second exchange: 17.5 against 16.1 us for 1 row of 32000).  The few
// tokens of the border's bin take one more.
template <bool BY_MASS, typename R>
__device__ __forceinline__ void narrow(const R& r, Kept& kept, unsigned long long want, float top_p) {
  SampleShared* s = r.s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, mine = threadIdx.x;
  int sh = 0;
  uint32_t kmax = 0, kmin = 0;
  const bool push = r.C > 1 && !BY_MASS;
  for (int level = 0;; level++) {
    // a surviving token's bin: of the row's range of logits, then of a range of keys
    auto bin = [&](float x) -> float { return level == 0 ? r.place(x) : (float)((kmax - key_of(x)) >> sh); };
    const float least = level == 0 ? kept.x : logit_of(kmin);
    auto inside = [&](float x, int i) -> bool {
      return x >= least && kept.has(x, i) && (level == 0 || key_of(x) <= kmax);
    };
    s->hist[0][mine] = s->hist[1][mine] = s->hist[2][mine] = 0;
    if (threadIdx.x == 0) s->filled = 0;
    __syncthreads();
    const uint32_t chunks = r.chunks(least);
    r.each(chunks, [&](int i, const float (&x)[4]) {
      uint32_t m = 0;
#pragma unroll
      for (int e = 0; e < 4; e++) m |= (inside(x[e], r.first + i + lane * 4 + e) ? 1u : 0u) << e;
      for (; m; m &= m - 1) {  // lanes take their tokens together, whichever of their four they are
        const float v = m & 1 ? x[0] : m & 2 ? x[1] : m & 4 ? x[2] : x[3];
        const int b = (int)bin(v);
        if (BY_MASS) add_mass(s, b, r.weight(v));
        else atomicAdd(&s->hist[0][b], 1u);
      }
    });
    if (push) {
      push_counts(r);
    } else if (r.C > 1) {
      __syncthreads();
      const unsigned long long sum = warp_sum(s->hist[1][mine] + ((unsigned long long)s->hist[2][mine] << 32));
      if (lane < (int)r.C) to_peer(&r.group[r.rank * GROUPS + warp], lane, sum);
    }
    row_sync(r);  // every CTA's histogram is complete
    int b;
    uint32_t n, ahead = 0;  // tokens of the border's bin, and of those in the CTAs before this one
    unsigned long long total, picked;
    if (BY_MASS && r.C > 1) {  // all warps alike
      unsigned long long sum = 0, inc;
      for (uint32_t c = 0; c < r.C; c++) sum += lane < GROUPS ? r.group[c * GROUPS + lane] : 0;
      inc = warp_scan(sum);
      total = __shfl_sync(ALL, inc, 31);
      if (level == 0) want = max(1ull, share_of<true>(total, top_p));
      if (total < want || total == 0) {  // all survivors (the same in every CTA)
        row_sync(r);                     // the sums have been read
        return;
      }
      const int g = __ffs(__ballot_sync(ALL, inc >= want)) - 1;
      want -= __shfl_sync(ALL, inc - sum, g);
      if (warp < (int)r.C) {
        const int at = g * 32 + lane;
        s->count[warp][lane] = from_peer(&s->hist[0][at], warp);
        s->mass[warp][lane] = from_peer(&s->hist[1][at], warp) + ((unsigned long long)from_peer(&s->hist[2][at], warp) << 32);
      }
      __syncthreads();
      uint32_t count = 0;
      sum = 0;
      for (uint32_t c = 0; c < r.C; c++) count += s->count[c][lane], sum += s->mass[c][lane];
      inc = warp_scan(sum);
      const int l = __ffs(__ballot_sync(ALL, inc >= want)) - 1;
      want -= __shfl_sync(ALL, inc - sum, l);
      n = __shfl_sync(ALL, count, l);
      picked = __shfl_sync(ALL, sum, l);
      b = g * 32 + l;
      ahead = warp_sum(lane < (int)r.rank ? s->count[lane % MAX_C][l] : 0u);
    } else {
      uint32_t count = 0;
      unsigned long long mass = 0;
      if (push) {
        for (uint32_t c = 0; c < r.C; c++) count += r.all[c * BINS + mine];
      } else {
        count = s->hist[0][mine];
        mass = s->hist[1][mine] + ((unsigned long long)s->hist[2][mine] << 32);
      }
      const unsigned long long v = BY_MASS ? mass : count;
      const unsigned long long before = block_scan(v, &total, s);
      if (level == 0 && BY_MASS) want = max(1ull, share_of<true>(total, top_p));
      if (total < want || total == 0) {  // all survivors (the same in every CTA)
        row_sync(r);                     // the counts have been read
        return;
      }
      if (before < want && want <= before + v) {
        s->pick = mine;
        s->pick_count = count;
        s->pick_mass = mass;
        s->before = before;
      }
      __syncthreads();
      b = s->pick;
      n = s->pick_count;
      picked = s->pick_mass;
      want -= s->before;
      if (push) ahead = warp_sum(lane < (int)r.rank ? r.all[lane * BINS + b] : 0u);
    }
    if (r.C > 1) cluster_arrive();  // the others' numbers have been read
    const uint32_t own = s->hist[0][b];
    if (n <= FEW) {
      // into every CTA's list, this CTA's behind those of the CTAs before it
      if (own)
        r.each(chunks, [&](int i, const float (&x)[4]) {
          const float most = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
          if (!__any_sync(ALL, most >= least && (level > 0 || r.place(most) < (float)(b + 1)))) return;
#pragma unroll
          for (int e = 0; e < 4; e++) {
            const int index = r.first + i + lane * 4 + e;
            if (!inside(x[e], index) || (int)bin(x[e]) != b) continue;
            const unsigned long long w = BY_MASS ? r.weight(x[e]) : 1;
            const Candidate* at = &s->few[ahead + atomicAdd(&s->filled, 1u)];
            for (uint32_t c = 0; c < r.C; c++)
              asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dsmem_addr(at, c)),
                           "r"(key_of(x[e])), "r"((uint32_t)index), "r"((uint32_t)w), "r"((uint32_t)(w >> 32))
                           : "memory");
          }
        });
      if (r.C > 1) cluster_wait();
      row_sync(r);
      // each token's sum of those before it; one of them is the last that is kept
      const uint32_t cand = threadIdx.x / 4;
      const bool one = cand < n;
      const Candidate me = s->few[one ? cand : 0];
      unsigned long long sum = 0;
      if (one)
        for (uint32_t k = threadIdx.x % 4; k < n; k += 4) {
          const Candidate o = s->few[k];
          if (o.key > me.key || (o.key == me.key && o.index < me.index)) sum += o.weight;
        }
      sum += __shfl_xor_sync(ALL, sum, 1);
      sum += __shfl_xor_sync(ALL, sum, 2);
      if (one && sum < want && want <= sum + me.weight) {
        s->pick_key = me.key;
        s->pick_index = me.index;
      }
      __syncthreads();
      kept.x = logit_of(s->pick_key);
      kept.index = (int)s->pick_index;
      __syncthreads();
      return;
    }
    // the range of the bin's keys
    if (r.C == 1) {
      uint32_t lo = ALL, hi = 0;
      for (uint32_t k = chunks; k; k &= k - 1) {
        const int i = r.w0 + (__ffs(k) - 1) * CHUNK;
        float x[4];
        r.four(i, x);
#pragma unroll
        for (int e = 0; e < 4; e++)
          if (inside(x[e], r.first + i + lane * 4 + e) && (int)bin(x[e]) == b) {
            lo = min(lo, key_of(x[e]));
            hi = max(hi, key_of(x[e]));
          }
      }
      lo = __reduce_min_sync(ALL, lo), hi = __reduce_max_sync(ALL, hi);
      if (lane == 0) s->warp_a[warp] = lo, s->warp_b[warp] = hi;
      __syncthreads();
      kmin = __reduce_min_sync(ALL, lane < SAMPLE_WARPS ? s->warp_a[lane] : ALL);
      kmax = __reduce_max_sync(ALL, lane < SAMPLE_WARPS ? s->warp_b[lane] : 0);
      __syncthreads();  // read by all warps: index_of writes its counts there
    } else {
      if (level == 0) {
        keys_of_bin(r, kept, b, &kmin, &kmax);
      } else {
        kmax -= (uint32_t)b << sh;
        if (kmax - kmin >> sh) kmin = kmax - ((1u << sh) - 1);
      }
      if (R::KEY_BITS == 16) {  // to the keys of 16-bit logits, which end in zeros, the negative ones' in ones
        kmax = kmax >> 31 ? kmax & ~0xFFFFu : kmax - ((kmax + 1) & 0xFFFFu);
        kmin = kmin >> 31 ? (kmin + 0xFFFFu) & ~0xFFFFu : kmin | 0xFFFFu;
        if (kmin == 0x7FFFFFFFu) kmin++;  // -0, which does not occur
      }
    }
    if (kmin == kmax) {  // one key: its first `want` by index
      if (BY_MASS) {
        const unsigned long long w = picked / n;  // they weigh the same
        want = w ? (want + w - 1) / w : n;
      }
      const float x = logit_of(kmax);
      int bound = x == kept.x ? kept.index : 0x7FFFFFFF;
      if (want < n) {  // the same in every CTA
        const uint32_t quota = want <= ahead ? 0 : want - ahead >= own ? own : (uint32_t)(want - ahead);
        if (quota < own) bound = index_of(r, kept, x, quota);
      }
      kept = {x, bound};
      if (r.C > 1) cluster_wait();
      __syncthreads();  // pick_index has been read
      return;
    }
    sh = r.C > 1 ? 32 - R::KEY_BITS : 0;
    while (((kmax - kmin) >> sh) >= (uint32_t)BINS) sh++;
    if (r.C > 1) cluster_wait();
    __syncthreads();  // pick has been read
  }
}

// Bytes of shared memory for all CTAs' counts and the list of survivors.
__host__ __device__ constexpr size_t shared_counts(int C) { return C == 1 ? 0 : (size_t)C * BINS * 4 + LIST * 8; }

// The first kept token, in order of the index, at which the running sum of
// the kept weights exceeds u times their sum.  `index`: the tokens' places in
// the row where they are not first + i.
template <typename R>
__device__ __forceinline__ void choose(const R& r, const Kept& kept, float min_p, float u, const uint32_t* index,
                                       int32_t* token, float* prob) {
  SampleShared* s = r.s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned long long least = 1;
  if (min_p > 0.f) least = max(1ull, share_of<true>(1ull << ONE_BITS, fminf(min_p, 1.f)));
  auto weights = [&](int i0, const float (&v)[4], unsigned long long (&w)[4]) -> unsigned long long {
    unsigned long long sum = 0;
    w[0] = w[1] = w[2] = w[3] = 0;
#pragma unroll
    for (int e = 0; e < 4; e++) {
      if (kept.has(v[e], r.first + i0 + lane * 4 + e)) w[e] = r.weight(v[e]);
      if (w[e] < least) w[e] = 0;
      sum += w[e];
    }
    return sum;
  };
  // the kept mass of each warp's tokens, of the CTAs, of the row
  unsigned long long mine = 0, w[4];
  const uint32_t chunks = r.chunks(kept.x);
  r.each(chunks, [&](int i, const float (&v)[4]) { mine += weights(i, v, w); });
  mine = warp_sum(mine);
  __syncthreads();  // warp_sum has been read
  if (lane == 0) s->warp_sum[warp] = mine;
  __syncthreads();
  const unsigned long long theirs = lane < SAMPLE_WARPS ? s->warp_sum[lane] : 0;
  unsigned long long before = warp_sum(lane < warp ? theirs : 0ull);
  unsigned long long total = warp_sum(theirs);
  if (r.C > 1) {
    if (threadIdx.x < r.C) to_peer(&s->peer[1][r.rank].sum, threadIdx.x, total);
    row_sync(r);
    const unsigned long long v = lane < (int)r.C ? s->peer[1][lane].sum : 0;
    before += warp_sum(lane < (int)r.rank ? v : 0ull);
    total = warp_sum(v);
  }
  unsigned long long target = u > 0.f ? share_of<false>(total, fminf(u, 1.f)) + 1 : 1;
  if (target > total) target = total;
  if (!(before < target && target <= before + mine)) return;
  for (uint32_t k = chunks; k && before < target; k &= k - 1) {
    const int i0 = r.w0 + (__ffs(k) - 1) * CHUNK;
    float v[4];
    r.four(i0, v);
    const unsigned long long sum = weights(i0, v, w);
    const unsigned long long inc = warp_scan(sum);
    if (before + inc >= target && before + inc - sum < target) {  // one lane
      unsigned long long run = before + inc - sum;
      int e = 0;
#pragma unroll
      for (int k = 0; k < 3; k++) {
        if (e == k && run + w[k] < target) run += w[k], e++;
      }
      const unsigned long long hit = e == 0 ? w[0] : e == 1 ? w[1] : e == 2 ? w[2] : w[3];
      const int i = i0 + lane * 4 + e;
      *token = index ? (int32_t)index[i] : r.first + i;
      if (prob) *prob = ratio(hit, total);
    }
    before += __shfl_sync(ALL, inc, 31);
  }
}

// Both filters and the choice over a list of `left` survivors in order of their
// index, `spread` places apart, four places per thread, which keeps their
// weights in registers.  One histogram of counts and masses serves both
// filters (one for each, and weights formed anew in every pass, took 3.4 us
// more).  False, with nothing written, where more than FEW tokens share the
// bin of a border.
template <typename R>
__device__ __forceinline__ bool finish(const R& r, const float* list_x, const uint32_t* list_index, uint32_t left, int spread,
                                       uint32_t top_k, float top_p, float min_p, float u, int32_t* token, float* prob) {
  static_assert(LIST == SAMPLE_THREADS * 4, "four places per thread");
  SampleShared* s = r.s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, mine = threadIdx.x;
  const float4 f = *reinterpret_cast<const float4*>(list_x + mine * 4);
  float v[4] = {f.x, f.y, f.z, f.w};
  unsigned long long w[4];
#pragma unroll
  for (int e = 0; e < 4; e++) {
    if (e % spread || mine * 4 + e >= (int)left * spread) v[e] = -INFINITY;
    w[e] = r.weight(v[e]);  // of -inf: 0
  }
  Kept kept = everything();
  if (left > top_k || top_p < 1.f) {
    s->hist[0][mine] = s->hist[1][mine] = s->hist[2][mine] = 0;
    if (mine == 0) s->filled = 0;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 4; e++)
      if (v[e] > -INFINITY) add_mass(s, (int)r.place(v[e]), w[e]);
    __syncthreads();
    const uint32_t count = s->hist[0][mine];
    const unsigned long long mass = s->hist[1][mine] + ((unsigned long long)s->hist[2][mine] << 32);
    uint32_t before = warp_scan(count);
    unsigned long long below = warp_scan(mass);
    if (lane == 31) s->warp_a[warp] = before, s->warp_sum[warp] = below;
    __syncthreads();
    const uint32_t counts = lane < SAMPLE_WARPS ? s->warp_a[lane] : 0;
    const unsigned long long masses = lane < SAMPLE_WARPS ? s->warp_sum[lane] : 0;
    before += warp_sum(lane < warp ? counts : 0u) - count;
    below += warp_sum(lane < warp ? masses : 0ull) - mass;
    unsigned long long total = warp_sum(masses), sum = 0, ahead = 0;
    const uint32_t cand = mine / 4;
    Candidate me = {};
    bool one = false;
    uint32_t rank = 0;
    // the bin's tokens, and for each the number and mass of those before it
    auto settle = [&](int b, uint32_t n) {
#pragma unroll
      for (int e = 0; e < 4; e++)
        if (v[e] > -INFINITY && (int)r.place(v[e]) == b)
          s->few[atomicAdd(&s->filled, 1u)] = {key_of(v[e]), (uint32_t)(mine * 4 + e), w[e]};
      __syncthreads();
      one = cand < n;
      me = s->few[one ? cand : 0];
      sum = 0, rank = 0;
      if (one)
        for (uint32_t k = mine % 4; k < n; k += 4) {
          const Candidate o = s->few[k];
          if (o.key > me.key || (o.key == me.key && o.index < me.index)) sum += o.weight, rank++;
        }
      sum += __shfl_xor_sync(ALL, sum, 1), rank += __shfl_xor_sync(ALL, rank, 1);
      sum += __shfl_xor_sync(ALL, sum, 2), rank += __shfl_xor_sync(ALL, rank, 2);
    };
    if (left > top_k) {
      if (before < top_k && top_k <= before + count) {
        s->pick = mine, s->pick_count = count, s->pick_index = before;
        s->before = below;
      }
      __syncthreads();
      const uint32_t n = s->pick_count, last = top_k - s->pick_index - 1;
      ahead = s->before;
      if (n > FEW) return false;
      settle(s->pick, n);
      if (one && rank == last) s->pick_key = me.key, s->pick_index = me.index, s->pick_mass = sum + me.weight;
      __syncthreads();
      kept = {logit_of(s->pick_key), (int)s->pick_index};
      total = ahead + s->pick_mass;
    }
    if (top_p < 1.f) {
      unsigned long long want = max(1ull, share_of<true>(total, fmaxf(top_p, 0.f)));
      __syncthreads();  // what was picked, and the list, have been read
      if (left > top_k && want > ahead) {
        want -= ahead;  // in the same bin
      } else {
        if (below < want && want <= below + mass) s->pick = mine, s->pick_count = count, s->before = below;
        if (mine == 0) s->filled = 0;
        __syncthreads();
        const uint32_t n = s->pick_count;
        want -= s->before;
        if (n > FEW) return false;
        settle(s->pick, n);
      }
      if (one && sum < want && want <= sum + me.weight) s->pick_key = me.key, s->pick_index = me.index;
      __syncthreads();
      kept = {logit_of(s->pick_key), (int)s->pick_index};
    }
  }
  unsigned long long least = 1, ours = 0;
  if (min_p > 0.f) least = max(1ull, share_of<true>(1ull << ONE_BITS, fminf(min_p, 1.f)));
#pragma unroll
  for (int e = 0; e < 4; e++) {
    if (!kept.has(v[e], mine * 4 + e) || w[e] < least) w[e] = 0;
    ours += w[e];
  }
  const unsigned long long upto = warp_scan(ours);
  if (lane == 31) s->warp_sum[warp] = upto;  // the scan's have been read, some barriers ago
  __syncthreads();
  const unsigned long long theirs = lane < SAMPLE_WARPS ? s->warp_sum[lane] : 0, all = warp_sum(theirs);
  unsigned long long run = warp_sum(lane < warp ? theirs : 0ull) + upto - ours;
  const unsigned long long target = min(all, u > 0.f ? share_of<false>(all, fminf(u, 1.f)) + 1 : 1);
  if (run < target && target <= run + ours) {  // one thread
    int e = 0;
#pragma unroll
    for (int k = 0; k < 3; k++)
      if (e == k && run + w[k] < target) run += w[k], e++;
    *token = (int32_t)list_index[mine * 4 + e];
    if (prob) *prob = ratio(e == 0 ? w[0] : e == 1 ? w[1] : e == 2 ? w[2] : w[3], all);
  }
  return true;
}

// One row per cluster of C CTAs.  STAGED: its logits are read once, into shared
// memory; else the chunks that a pass needs are read again where they are,
// mostly from L2, so that slices of 65536 tokens leave room for two CTAs per SM.
// Bound by latency, not by the bytes (0.6 us for 8 rows of 131071): reading
// (2 us), the exchanges between the CTAs (1 to 2 us each with 16 CTAs), and
// passes over 4 to 64 tokens per thread; for many rows by the instructions of
// those passes.  Measured: 8 rows of 131071, all filters, 12.0 us; 1 row of
// 32000, top-p, 15.4 us; 64 rows of 262144 in bf16, top-k and top-p, 29.2 us;
// top-p alone has to weigh every token: 1 row of 131071, 32 us.
template <typename T, bool STAGED>
__global__ void __launch_bounds__(SAMPLE_THREADS, 2) qlin_sample_kernel(const __grid_constant__ SampleParams p, int C) {
  extern __shared__ __align__(16) uint8_t raw[];
  SampleShared* s = reinterpret_cast<SampleShared*>(raw);
  uint32_t* all = reinterpret_cast<uint32_t*>(raw + sizeof(SampleShared));
  float* list_x = reinterpret_cast<float*>(all + C * BINS);
  uint32_t* list_index = reinterpret_cast<uint32_t*>(list_x + LIST);
  T* x = reinterpret_cast<T*>(raw + sizeof(SampleShared) + shared_counts(C));
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Row<T, STAGED ? 16 : 32, STAGED> r;  // a slice of 32768 or 65536 tokens at most (STAGED_SLICE, IN_PLACE_SLICE)
  r.s = s;
  r.all = all;
  r.group = reinterpret_cast<unsigned long long*>(list_x);  // a list of survivors has no use for it
  r.C = C;
  r.rank = C == 1 ? 0 : cluster_ctarank();
  r.first = (int)(r.rank * p.slice);
  const int row = blockIdx.x / C;
  const int tokens = max(0, min(p.slice, p.V - r.first));
  r.part(p.slice);
  if (C > 1) cluster_arrive_relaxed();
  if (threadIdx.x < 32) s->table[threadIdx.x] = TABLE[threadIdx.x];
  pdl_wait();
  pdl_launch_dependents();
  const float temperature = p.temperature ? p.temperature[row] : 1.f;
  const int top_k = p.top_k ? p.top_k[row] : 0;
  const float top_p = p.top_p ? p.top_p[row] : 1.f;
  const float min_p = p.min_p ? p.min_p[row] : 0.f;
  const float u = p.u[row];
  const T* src = static_cast<const T*>(p.logits) + row * p.ld + r.first;
  r.tokens = tokens;
  r.wide = (reinterpret_cast<uintptr_t>(src) & (4 * sizeof(T) - 1)) == 0;
  r.inf = false;
  // Of four tokens at a time only the largest counts for now: an instruction or
  // two per token (looking at each for the least and the first of the largest
  // made it 15).
  float mx = -INFINITY, mn = INFINITY;  // the largest, NaN if one is; the least of the largest of four
  auto look = [&](int c, const float (&v)[4]) {
    const float t = max_of(v);
    r.set_top(c, t);
    mx = max_of(mx, t);
    if (t > -INFINITY) mn = fminf(mn, t);
  };
  constexpr int CHUNKS = STAGED ? 16 : 32;
  if (!STAGED || (r.wide && sizeof(T) == 2)) {  // (fp32 is staged faster by single words: 8 rows of 524288 28.5 against 22.4 us)
    r.x = STAGED ? x : src;
    constexpr int BATCH = sizeof(T) == 4 ? 2 : STAGED ? 16 : 4;  // more spill registers
#pragma unroll
    for (int c0 = 0; c0 < CHUNKS; c0 += BATCH) {
      typename decltype(r)::Four f[BATCH];
#pragma unroll
      for (int k = 0; k < BATCH; k++)
        if (r.w0 + (c0 + k) * CHUNK < r.w1) f[k] = r.fetch(src, r.w0 + (c0 + k) * CHUNK);
#pragma unroll
      for (int k = 0; k < BATCH; k++) {
        const int i = r.w0 + (c0 + k) * CHUNK;
        r.no_top(c0 + k);
        if (i < r.w1) {
          if constexpr (STAGED) *reinterpret_cast<typename decltype(r)::Four*>(x + i + lane * 4) = f[k];
          float v[4];
          r.values(f[k], v);
          look(c0 + k, v);
        }
      }
    }
    __syncwarp();
  } else {
    r.x = x;
    constexpr int BATCH = 16;  // loads in flight per thread
    for (int i0 = r.w0 + lane; i0 < r.w1; i0 += 32 * BATCH) {
      T v[BATCH];
#pragma unroll
      for (int k = 0; k < BATCH; k++) v[k] = i0 + 32 * k < tokens ? src[i0 + 32 * k] : T(-INFINITY);
#pragma unroll
      for (int k = 0; k < BATCH; k++)
        if (i0 + 32 * k < r.w1) x[i0 + 32 * k] = v[k];
    }
    __syncwarp();
#pragma unroll
    for (int c = 0; c < CHUNKS; c++) {
      r.no_top(c);
      if (r.w0 + c * CHUNK < r.w1) {
        float v[4];
        r.four(r.w0 + c * CHUNK, v);
        look(c, v);
      }
    }
  }
  uint32_t nan = mx != mx, top = ALL;  // top: the lowest index of the largest, if that is the answer
  if (!(temperature > 0.f)) {
#pragma unroll 1
    for (int i = r.w0; i < r.w1; i += CHUNK) {
      float v[4];
      r.four(i, v);
#pragma unroll
      for (int e = 0; e < 4; e++)
        if (v[e] == mx) top = min(top, (uint32_t)(r.first + i + lane * 4 + e));
    }
  }
  // of the warp, the CTA, the row, as keys; the index of the largest
  uint32_t kmx = key_of(mx), kmn = key_of(mn);
  auto join = [&](bool in) {
    const uint32_t best = __reduce_max_sync(ALL, in ? kmx : 0);
    top = __reduce_min_sync(ALL, in && kmx == best ? top : ALL);
    kmx = best;
    kmn = __reduce_min_sync(ALL, in ? kmn : ALL);
    nan = __any_sync(ALL, in && nan);
  };
  // A logit that top_k tokens reach at least: each of the row's warps with a
  // full part gives the j-th of its 32 lanes' largest tokens, and the
  // ceil(top_k / j)-th of these is reached by j tokens in as many warps.  With j
  // about top_k over the warps, some 1.8 top_k tokens of normally distributed
  // logits reach it (the least of all warps' would be reached by 3 to 40 top_k).
  const uint32_t full = (uint32_t)p.V / (uint32_t)(r.w1 - r.w0);
  const uint32_t per_warp = C > 1 && top_k > 0 && top_k < p.V && full ? top_k / full + 1 : 33;
  uint32_t reach = 0;
  if (per_warp <= 32 && r.w1 <= tokens) {
    uint32_t key = kmx;
    for (uint32_t j = 0; j < per_warp; j++) {
      reach = __reduce_max_sync(ALL, key);
      if (lane == __ffs(__ballot_sync(ALL, key == reach)) - 1) key = 0;
    }
  }
  join(true);
  if (lane == 0) {
    s->warp_a[warp] = nan, s->warp_b[warp] = top, s->warp_c[warp] = kmx, s->warp_d[warp] = kmn;
    if (C > 1) s->reach[r.rank * SAMPLE_WARPS + warp] = reach;
  }
  __syncthreads();
  const int from = lane % SAMPLE_WARPS;
  nan = s->warp_a[from], top = s->warp_b[from], kmx = s->warp_c[from], kmn = s->warp_d[from];
  join(true);
  if (C > 1) {
    cluster_wait();  // every CTA of the row has started
    if (threadIdx.x < C) {
      const Round* at = &s->peer[0][r.rank];
      to_peer(&at->kmx, threadIdx.x, kmx);
      to_peer(&at->kmn, threadIdx.x, kmn);
      to_peer(&at->nan, threadIdx.x, nan);
      to_peer(&at->top, threadIdx.x, top);
    }
    if (per_warp <= 32 && threadIdx.x < C * SAMPLE_WARPS) {
      const uint32_t c = threadIdx.x / SAMPLE_WARPS;
      const uint32_t* at = &s->reach[r.rank * SAMPLE_WARPS + threadIdx.x % SAMPLE_WARPS];
      if (c != r.rank) to_peer(at, c, *at);
    }
    row_sync(r);
    if (lane < C) {
      const Round o = s->peer[0][lane];
      kmx = o.kmx, kmn = o.kmn, nan = o.nan, top = o.top;
    }
    join(lane < C);
  }
  mx = logit_of(kmx), mn = logit_of(kmn);
  if (nan || mx == -INFINITY || !(temperature > 0.f)) {  // no token, or the largest
    const bool none = nan || mx == -INFINITY;
    if (r.rank == 0 && threadIdx.x == 0) {
      p.token[row] = none ? -1 : (int32_t)top;
      if (p.prob) p.prob[row] = none ? 0.f : 1.f;
    }
    return;
  }
  float low = -INFINITY;
  if (per_warp <= 32) {  // by bisection of the keys' leading halves (what is cut off lowers it), alike in all warps
    const uint32_t need = (top_k + per_warp - 1) / per_warp;
    uint32_t keys[MAX_C * SAMPLE_WARPS / 32], lo = ALL, hi = 0;
#pragma unroll
    for (int k = 0; k < MAX_C * SAMPLE_WARPS / 32; k++) {
      keys[k] = lane + 32 * k < C * SAMPLE_WARPS ? s->reach[lane + 32 * k] >> 16 : 0;
      lo = min(lo, keys[k] ? keys[k] : ALL), hi = max(hi, keys[k]);
    }
    lo = __reduce_min_sync(ALL, lo), hi = __reduce_max_sync(ALL, hi);
    while (lo < hi) {
      const uint32_t mid = hi - (hi - lo) / 2;
      uint32_t n = 0;
#pragma unroll
      for (int k = 0; k < MAX_C * SAMPLE_WARPS / 32; k++) n += keys[k] >= mid ? 1 : 0;
      if (__reduce_add_sync(ALL, n) >= need) lo = mid;
      else hi = mid - 1;
    }
    if (lo > key_of(-INFINITY) >> 16) low = logit_of(lo << 16);
  }
  if (mx == INFINITY) {  // the infinite ones are left, alike
    if constexpr (STAGED) {
      __syncwarp();
      for (int i = r.w0 + lane; i < r.w1; i += 32) x[i] = to_float(x[i]) == INFINITY ? T(0.f) : T(-INFINITY);
      __syncwarp();
    } else {
      r.inf = true;
    }
    r.tops();
    mx = mn = low = 0.f;
  }
  if (low > -INFINITY) mn = low;  // the bins divide what lies above
  r.mx = mx, r.mn = fmaxf(low, -FLT_MAX);
  r.weighing = weighing(mx, temperature);
  r.to_bin = mx - mn > 0.f ? fminf((float)(BINS - 1) / (mx - mn), 3e38f) : 0.f;

  Kept kept = low > -INFINITY ? Kept{low, 0x7FFFFFFF} : everything();
  if (top_k > 0 && top_k < p.V) {
    if (C > 1 && top_k <= LIST / 2) {
      // The tokens that reach `low` (without one, those that are not
      // forbidden): if few, the first CTA of the row goes on alone with them.
      // (An exchange between the CTAs costs more than a pass over a list.)
      // Each warp lays down its own, then the CTAs' numbers give their places.
      uint2* own = reinterpret_cast<uint2*>(s->hist) + warp * OWN;
      static_assert(offsetof(SampleShared, count) >= SAMPLE_WARPS * OWN * sizeof(uint2), "hist and mass hold the lists");
      const float least = fmaxf(low, -FLT_MAX);
      uint32_t n = 0;
      r.each(r.chunks(least), [&](int i, const float (&v)[4]) {
        uint32_t at = n;
        const uint32_t ahead = (1u << lane) - 1;
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const uint32_t them = __ballot_sync(ALL, v[e] >= least);
          at += __popc(them & ahead);
          n += __popc(them);
        }
#pragma unroll
        for (int e = 0; e < 4; e++)
          if (v[e] >= least) {
            if (at < OWN) own[at] = make_uint2(__float_as_uint(v[e]), (uint32_t)(r.first + i + lane * 4 + e));
            at++;
          }
      });
      if (lane == 0) s->warp_a[warp] = n <= OWN ? n : LIST + 1;
      __syncthreads();
      const uint32_t theirs = lane < SAMPLE_WARPS ? s->warp_a[lane] : 0;
      uint32_t at = warp_sum(lane < warp ? theirs : 0u);
      const uint32_t ours = warp_sum(theirs);
      if (threadIdx.x < C) to_peer(&s->peer[0][r.rank].left, threadIdx.x, ours);
      row_sync(r);
      const uint32_t m = lane < C ? s->peer[0][lane].left : 0;
      const uint32_t left = warp_sum(m);
      at += warp_sum(lane < (int)r.rank ? m : 0u);
      if (left <= LIST) {
        // in order of their index; fewer than half a lane's four places each
        // leave gaps, so that all warps have their share
        int spread = 1;
        while (spread < 4 && left * spread * 2 <= CHUNK * SAMPLE_WARPS) spread *= 2;
        for (uint32_t t = lane; t < n; t += 32) {
          to_peer(&list_x[(at + t) * spread], 0, own[t].x);
          to_peer(&list_index[(at + t) * spread], 0, own[t].y);
        }
        row_sync(r);
        if (r.rank) return;
        int32_t* const token = p.token + row;
        float* const prob = p.prob ? p.prob + row : nullptr;
        if (finish(r, list_x, list_index, left, spread, (uint32_t)top_k, top_p, min_p, u, token, prob)) return;
        __syncthreads();
        Row<float, LIST / (CHUNK * SAMPLE_WARPS)> one;
        one.x = list_x;
        one.s = s;
        one.all = nullptr;
        one.C = 1;
        one.rank = 0;
        one.first = 0;
        one.part((int)left * spread);
        one.mx = r.mx, one.to_bin = r.to_bin, one.weighing = r.weighing;
        const int room = (one.w1 - one.w0) * SAMPLE_WARPS;
        for (int i = threadIdx.x; i < room; i += SAMPLE_THREADS)
          if (i % spread || i >= (int)left * spread) list_x[i] = -INFINITY;
        __syncthreads();
        one.tops();
        kept = everything();
        if (left > (uint32_t)top_k) narrow<false>(one, kept, (unsigned long long)top_k, 0.f);
        if (top_p < 1.f) narrow<true>(one, kept, 0, fmaxf(top_p, 0.f));
        choose(one, kept, min_p, u, list_index, token, prob);
        return;
      }
    }
    narrow<false>(r, kept, (unsigned long long)top_k, 0.f);
  }
  if (top_p < 1.f) narrow<true>(r, kept, 0, fmaxf(top_p, 0.f));
  choose(r, kept, min_p, u, nullptr, p.token + row, p.prob ? p.prob + row : nullptr);
}

constexpr int STAGED_SLICE = 32768;  // tokens of a slice in shared memory at most
constexpr int IN_PLACE_SLICE = 65536;
constexpr size_t SAMPLE_SMEM = 220 * 1024;
static_assert(sizeof(SampleShared) + shared_counts(MAX_C) + STAGED_SLICE * 4 <= SAMPLE_SMEM, "largest slice");
static_assert(MAX_C * STAGED_SLICE >= QLIN_SAMPLE_MAX_V && 8 * IN_PLACE_SLICE >= QLIN_SAMPLE_MAX_V, "the longest row");

const void* sample_fn(int dtype, bool staged) {
  if (dtype == QLIN_F32)
    return staged ? reinterpret_cast<const void*>(qlin_sample_kernel<float, true>)
                  : reinterpret_cast<const void*>(qlin_sample_kernel<float, false>);
  return staged ? reinterpret_cast<const void*>(qlin_sample_kernel<__nv_bfloat16, true>)
                : reinterpret_cast<const void*>(qlin_sample_kernel<__nv_bfloat16, false>);
}

struct SamplePlan {
  int C;  // CTAs per row, a power of two
  bool staged;
};

// Slices of 64 KB in shared memory leave room for two CTAs per SM.  Few rows
// take more CTAs each: a pass costs less, an exchange more.  Under top-k the
// passes are over few tokens: up to 128 CTAs (8 rows of 131071: 4, 8 and 16
// CTAs per row 13.9, 12.0 and 13.9 us; 64 rows of 32000 with 2 and 4: 13.0 and
// 14.0), clusters of 16 for four rows at most (4 rows of 262144 with 8 and 16:
// 13.2 and 12.2; 1 row of 32000: 10.1 and 10.8).  Else all tokens are weighed:
// up to 256 CTAs (32 rows of 32000 with 4 and 8: 30.6 and 26.3; 64 rows with 4
// and 8: 38.5 and 45.1), and clusters of 16 while their slices are large
// beside the rows' number (16 rows of 131071 with 8 and 16: 53.0 and 48.2; of
// 32000: 22.3 and 27.7).  From 16384 tokens on two CTAs pay for any number of
// rows (256 rows of 32000 in bf16 with 1 and 2: 65 and 30 us).
// Clusters of 16, of which few fit at a time, are worth avoiding: by slices of
// 128 KB while one wave of them does (16 rows of 262144 in fp32 under top-k
// with 16 and 8 CTAs: 25.6 and 19.9), else by reading the rows where they are
// (64 rows of 262144 in fp32 under top-k with 16 staged and 4 such CTAs: 76.2
// and 34.9; 32 rows under top-p with 16 and 8: 200 and 145).  With 8 that pays
// for many fp32 rows under top-k (128 rows of 131071 with 8 and 2: 49.2 and
// 40.9; 48 rows with 8 and 4: 25.6 and 26.3), not for bf16 (64 rows of 262144
// with 8 and 4: 29.5 and 33.0) or top-p (203 and 258).
SamplePlan sample_plan(int64_t M, int64_t V, int64_t size, bool by_count, int most) {
  constexpr int64_t SMS = 152;
  int C = V > 16384 ? 2 : 1;
  while (C < most && C * (int64_t)65536 < V * size) C *= 2;
  if (V > C * (int64_t)STAGED_SLICE) return {8, false};  // where clusters of 16 do not fit the device
  if (by_count && C == 16 && V <= 8 * 32768 && M > 4 && 8 * M <= SMS) return {8, true};
  if (by_count ? C == 16 ? M > 8 : C == 8 && size == 4 && M >= 64 : C == 16 && C * M > 2 * SMS) {
    for (C = 2; C * (int64_t)IN_PLACE_SLICE < V;) C *= 2;
    while (C < 8 && 2 * C * M <= 2 * SMS) C *= 2;
    return {C, false};
  }
  while (C < 8 && C * (int64_t)(SAMPLE_THREADS * 4) < V && 2 * C * M <= (by_count ? 128 : 256)) C *= 2;
  if (C == 8 && most == 16 && (by_count ? M <= 4 && V >= 65536 : M <= 16 && V > 16384 && V >= 2048 * M)) C = 16;
  return {C, true};
}

struct SampleDevice {
  std::once_flag once;
  qlin_status ready = QLIN_ERR_CUDA;
  int most = 8;  // CTAs of a cluster
};
SampleDevice g_sample[64];

// The kernels' attributes, and whether the device holds clusters of 16 with the
// largest slice, once per device.
qlin_status sample_setup(int* most) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return status_of(e);
  if (dev < 0 || dev >= 64) return QLIN_ERR_CUDA;
  SampleDevice& d = g_sample[dev];
  std::call_once(d.once, [&d] {
    cudaError_t e = cudaSuccess;
    int clusters = 1;
    for (int dtype : {QLIN_F32, QLIN_BF16}) {
      for (bool staged : {true, false}) {
        if (e == cudaSuccess)
          e = cudaFuncSetAttribute(sample_fn(dtype, staged), cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SAMPLE_SMEM);
        if (e == cudaSuccess)
          e = cudaFuncSetAttribute(sample_fn(dtype, staged), cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      }
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(MAX_C, 1, 1);
      cfg.blockDim = dim3(SAMPLE_THREADS, 1, 1);
      cfg.dynamicSmemBytes = SAMPLE_SMEM;
      cudaLaunchAttribute attr;
      attr.id = cudaLaunchAttributeClusterDimension;
      attr.val.clusterDim.x = MAX_C;
      attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
      cfg.attrs = &attr;
      cfg.numAttrs = 1;
      int n = 0;
      if (e == cudaSuccess && cudaOccupancyMaxActiveClusters(&n, sample_fn(dtype, true), &cfg) != cudaSuccess) {
        (void)cudaGetLastError();
        n = 0;
      }
      if (n < clusters) clusters = n;
    }
    if (clusters > 0) d.most = MAX_C;
    d.ready = status_of(e);
  });
  *most = d.most;
  return d.ready;
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
  int most = 0;
  qlin_status st = sample_setup(&most);
  if (st != QLIN_OK) return st;
  const SamplePlan plan = sample_plan(M, V, dtype == QLIN_F32 ? 4 : 2, top_k != nullptr, most);
  const int C = plan.C;
  SampleParams p = {logits, ld, u, temperature, top_p, min_p, top_k, token, prob, (int)V,
                    (int)(((V + C - 1) / C + CHUNK * SAMPLE_WARPS - 1) / (CHUNK * SAMPLE_WARPS) * (CHUNK * SAMPLE_WARPS))};
  int c = C;
  void* args[] = {&p, &c};
  const size_t slice = plan.staged ? (size_t)p.slice * (dtype == QLIN_F32 ? 4 : 2) : 0;
  return launch_step(sample_fn(dtype, plan.staged), dim3((unsigned)(M * C), 1, 1), dim3(SAMPLE_THREADS, 1, 1),
                     sizeof(SampleShared) + shared_counts(C) + slice, static_cast<cudaStream_t>(stream), args,
                     (flags & QLIN_FLAG_PDL) != 0, C);
}

extern "C" qlin_status qlin_debug_sample_weight(int n, const float* x, const float* max, const float* temperature,
                                                uint64_t* weight) {
  static const uint32_t table[32] = QLIN_EXP2_TABLE;
  if (n < 0 || (n && (!x || !max || !temperature || !weight))) return QLIN_ERR_INVALID_ARG;
  for (int i = 0; i < n; i++)
    if (!(x[i] <= max[i]) || !std::isfinite(max[i]) || !(temperature[i] > 0.f)) return QLIN_ERR_INVALID_ARG;
  for (int i = 0; i < n; i++) weight[i] = weight_of(x[i], weighing(max[i], temperature[i]), table);
  return QLIN_OK;
}

extern "C" qlin_status qlin_debug_sample_plan(int64_t M, int64_t V, int dtype, int top_k, int most, int* ctas,
                                              int* in_place) {
  if (M < 1 || M > (1 << 24) || V < 1 || V > QLIN_SAMPLE_MAX_V || (dtype != QLIN_F32 && dtype != QLIN_BF16) ||
      (top_k != 0 && top_k != 1) || (most != 8 && most != MAX_C) || !ctas || !in_place)
    return QLIN_ERR_INVALID_ARG;
  const SamplePlan plan = sample_plan(M, V, dtype == QLIN_F32 ? 4 : 2, top_k != 0, most);
  *ctas = plan.C;
  *in_place = plan.staged ? 0 : 1;
  return QLIN_OK;
}
