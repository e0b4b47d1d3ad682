// The integer weights of qlin_sample: exp((x - max) / T) as a multiple of
// 2^-42.  The same source on the device (the kernel) and on the host (the test
// export): every operation in it rounds alike on both.
#pragma once
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

namespace qlin {

#define QLIN_HD __host__ __device__ __forceinline__

constexpr int ONE_BITS = 42;  // weights are multiples of 2^-42; 2^19 of them sum below 2^62

// 2^(i/32) in units of 2^-31, to the nearest
#define QLIN_EXP2_TABLE                                                                                     \
  {0x80000000u, 0x82CD8699u, 0x85AAC368u, 0x88980E81u, 0x8B95C1E4u, 0x8EA4398Bu, 0x91C3D374u, 0x94F4EFA9u,  \
   0x9837F052u, 0x9B8D39BAu, 0x9EF53261u, 0xA2704303u, 0xA5FED6AAu, 0xA9A15AB5u, 0xAD583EEAu, 0xB123F582u,  \
   0xB504F334u, 0xB8FBAF47u, 0xBD08A39Fu, 0xC12C4CCAu, 0xC5672A11u, 0xC9B9BD86u, 0xCE248C15u, 0xD2A81D92u,  \
   0xD744FCCBu, 0xDBFBB798u, 0xE0CCDEECu, 0xE5B906E7u, 0xEAC0C6E8u, 0xEFE4B99Cu, 0xF5257D15u, 0xFA83B2DBu}

QLIN_HD uint32_t mul_high(uint32_t a, uint32_t b) {
#ifdef __CUDA_ARCH__
  return __umulhi(a, b);
#else
  return (uint32_t)(((uint64_t)a * b) >> 32);
#endif
}
QLIN_HD long long round_to_int(float x) {  // half to even
#ifdef __CUDA_ARCH__
  return __float2ll_rn(x);
#else
  return llrintf(x);
#endif
}
QLIN_HD int round_to_int32(float x) {
#ifdef __CUDA_ARCH__
  return __float2int_rn(x);
#else
  return (int)lrintf(x);
#endif
}

// What weight_of takes for a row: its logits times `scale` (a half where the
// difference of two finite ones may pass the largest float, else one), and
// log2(e) / (T scale) as a pair of floats: the quotient of the leading part,
// and that of what is left.  T above 0; an infinite one gives zeros.
struct Weighing {
  float scale, mx, ch, cl;
};
QLIN_HD Weighing weighing(float mx, float T) {
  constexpr float E_HI = 1.44269502f, E_LO = (float)(1.44269504088896341 - (double)E_HI);
  const float scale = mx >= 0x1p100f ? 0.5f : 1.f, c = E_HI / T;
  const float cl = c == 0.f ? 0.f : (fmaf(-c, T, E_HI) + E_LO) / T;
  return {scale, mx * scale, c / scale, cl / scale};
}

// exp((x - max) / T).  With c = log2(e) / T as a pair of floats, y = (x - max) c
// is formed to about 2^-40 (of temperatures up to 2^100; beyond, the pair comes
// to the last bits of its range), split into integer part and a 32-bit
// fraction f; 2^f is a table of 2^(i/32) times the series of e^z, z < ln(2)/32
// (table and short series: Tang, "Table-driven implementation of the
// exponential function", 1989), its first-order term in integers and the rest,
// below 2^-12, in fp32.  (The scale costs 0.15 of 15.2 us for 1 row of 32000
// under top-p; a way of their own for differences past the range cost 0.35.)
QLIN_HD unsigned long long weight_of(float logit, const Weighing& r, const uint32_t* table) {
  const float x = logit * r.scale, mx = r.mx, ch = r.ch, cl = r.cl;
  const float d = x - mx;
  if (!(d < 0.f)) return d == 0.f ? 1ull << ONE_BITS : 0;  // the largest; NaN cannot come here
  const float t = d - x;
  const float e = (x - (d - t)) + (-mx - t);  // d + e = x - mx exactly
  const float yh = d * ch;
  if (!(yh > -(ONE_BITS + 2.f))) return 0;  // below half a unit (-inf too)
  const float yl = fmaf(d, ch, -yh) + fmaf(d, cl, e * ch);
  const long long fix = round_to_int(yh * 4294967296.f) + round_to_int32(yl * 4294967296.f);
  if (fix >= 0) return 1ull << ONE_BITS;  // yh = 0 and a correction that rounds to it
  const uint32_t f = (uint32_t)fix;
  const int shift = -(int)(fix >> 32);  // >= 1
  const uint32_t z = mul_high(f << 5, 0xB17217F8u);  // (f mod 1/32) ln 2, in units of 2^-37
  const float zf = (float)z * 0x1p-37f;
  const uint32_t em1 = z + (uint32_t)(zf * zf * fmaf(zf, fmaf(zf, 1.f / 24, 1.f / 6), 0.5f) * 0x1p37f);  // e^z - 1
  const uint32_t base = table[f >> 27];
  const uint32_t m = base + (mul_high(base, em1) >> 5);  // 2^f in units of 2^-31
  return shift > ONE_BITS + 1 ? 0 : ((((unsigned long long)m << (ONE_BITS - 31 + 1)) >> shift) + 1) >> 1;
}

}  // namespace qlin
