// Rows of 8-bit integers: scale = m / 127 and q = 127 x / m rounded to the nearest integer, exact halves to the even one,
// with m the largest |x| of the row.  (quantize.cu, linear_int8.cu, residual_norm.cu)
#pragma once

#include "common.cuh"

namespace sesg {

// What the elements of a row share.  m is found as the largest bit pattern of |x|: infinities and NaN come out on top.
struct RowScale {
  float step;    // 127 / m: x * step is within 2e-5 of the quotient
  float limit;   // quotients nearer than 0.5 - limit to a half are decided exactly; -1: all of them
  float pre, a;  // 2^-e, and m 2^-e, which is below 2 (1 <= ... unless m is subnormal)
  float scale;   // m / 127
  int ok;        // finite
};

__device__ __forceinline__ RowScale row_scale(uint32_t most) {
  RowScale s;
  s.ok = most < 0x7f800000u;
  const float m = __uint_as_float(most);
  const uint32_t e = most >> 23 ? most >> 23 : 1;
  s.pre = __uint_as_float(e >= 254 ? 0x00400000u : (254 - e) << 23);
  s.a = m * s.pre;
  // 127 / m would be infinite below 2^-121: those rows are scaled first
  const bool tiny = m < 1e-35f;
  s.step = !s.ok || most == 0 || tiny ? 0.f : 127.f / m;
  s.limit = tiny ? -1.f : 0.4999f;
  s.scale = s.ok ? m / 127.f : __uint_as_float(0x7fc00000u);
  return s;
}

// q of one element, exactly: whether 127 x is above or below a half-integer times m, by products whose rounding errors are
// kept (two fused multiply-adds; the differences of the rounded products are exact, since those are within a factor of two).
static __device__ __noinline__ int quantize_exact(float x, float pre, float a) {
  if (a == 0.f) return 0;
  const float v = x * pre;
  const float lo = floorf(v * (127.f / a)), half = lo + 0.5f;
  const float p = v * 127.f, pe = fmaf(v, 127.f, -p), h = half * a, he = fmaf(half, a, -h);
  const float over = (p - h) + (pe - he);
  const int l = (int)lo;
  return over > 0.f ? l + 1 : over < 0.f ? l : l + (l & 1);
}

constexpr float kRoundMagic = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer, halves to even

// Eight neighbouring elements -> eight bytes.  x * step lies within 2e-5 of the quotient, so that only quotients within
// 1e-4 of a half need the exact decision (in 16 bits many are one exactly, x = m / 2 among them).
__device__ __forceinline__ uint2 quantize8(const float (&x)[8], const RowScale& s) {
  if (!s.ok) return make_uint2(0, 0);
  float t[8], off = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    t[i] = fmaf(x[i], s.step, kRoundMagic);
    off = fmaxf(off, fabsf(fmaf(x[i], s.step, kRoundMagic - t[i])));
  }
  if (off > s.limit) {
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = __int_as_float(quantize_exact(x[i], s.pre, s.a));
  }
  uint2 r;
  r.x = __byte_perm(__byte_perm(__float_as_uint(t[0]), __float_as_uint(t[1]), 0x0040),
                    __byte_perm(__float_as_uint(t[2]), __float_as_uint(t[3]), 0x0040), 0x5410);
  r.y = __byte_perm(__byte_perm(__float_as_uint(t[4]), __float_as_uint(t[5]), 0x0040),
                    __byte_perm(__float_as_uint(t[6]), __float_as_uint(t[7]), 0x0040), 0x5410);
  return r;
}

// Eight 16-bit elements as fp32.
__device__ __forceinline__ void unpack8(const uint4& v, int bf16, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (bf16) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

__device__ __forceinline__ void unpack8(const uint4& a, const uint4& b, float (&x)[8]) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
}

// The larger of two pairs of 16-bit |x| patterns, without signs.
__device__ __forceinline__ uint32_t most16(uint32_t m, uint32_t v) { return __vmaxu2(m, v & 0x7fff7fffu); }
__device__ __forceinline__ uint32_t most16(uint32_t m, const uint4& v) {
  return most16(most16(most16(most16(m, v.x), v.y), v.z), v.w);
}
__device__ __forceinline__ uint32_t most32(uint32_t m, const uint4& v) {
  return max(max(max(m, v.x & 0x7fffffffu), max(v.y & 0x7fffffffu, v.z & 0x7fffffffu)), v.w & 0x7fffffffu);
}
// ... its larger half as the pattern of the same value in fp32
__device__ __forceinline__ uint32_t most_f32(uint32_t m, int bf16) {
  const uint32_t h = max(m & 0xffffu, m >> 16);
  return bf16 ? h << 16 : __float_as_uint(__half2float(__ushort_as_half((unsigned short)h)));
}
__device__ __forceinline__ uint32_t warp_most(uint32_t m) { return __reduce_max_sync(0xffffffffu, m); }

// Four 8-bit integers as fp16: q + 128 in the mantissa of 1024, less 1152.
__device__ __forceinline__ void to_f16(uint32_t w, uint32_t& a, uint32_t& b) {
  const uint32_t u = w ^ 0x80808080u;
  const __half2 bias = __half2half2(__ushort_as_half(0x6480));
  uint32_t lo = __byte_perm(u, 0x64646464u, 0x4140), hi = __byte_perm(u, 0x64646464u, 0x4342);
  const __half2 l = __hsub2(*reinterpret_cast<__half2*>(&lo), bias), h = __hsub2(*reinterpret_cast<__half2*>(&hi), bias);
  a = *reinterpret_cast<const uint32_t*>(&l);
  b = *reinterpret_cast<const uint32_t*>(&h);
}

// A product's value from its integer sum and scales.  (Rounded one by one, so that every kernel gives the same bits.)
__device__ __forceinline__ float int8_value(int sum, float x_scale, float w_scale, float bias) {
  return __fadd_rn(__fmul_rn((float)sum, __fmul_rn(x_scale, w_scale)), bias);
}

}  // namespace sesg
