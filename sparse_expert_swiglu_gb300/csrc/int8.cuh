// Rows of 8-bit integers: scale = m / 127 and q = 127 x / m rounded to the nearest integer, exact halves to the even one,
// with m the largest |x| of the row.  (quantize.cu, linear_int8.cu, residual_norm.cu)
#pragma once

#include "common.cuh"

namespace sesg {

// What the elements of a row share.  m is found as the largest bit pattern of |x|: infinities and NaN come out on top.
//
// A row of 16-bit values takes no more than a product for each element.  With x and m integers X, Y below 2^11 times powers of
// two, a quotient that is no half is at least 1 / (2 Y) >= 2^-12 away from one, and 127 x / m is a half only where 127 divides
// 2 k + 1, at 63.5, which goes to the even 64, or Y.  So step, 127 / m or up to 2^-23 of it above, rounds every quotient
// right (127 * 2^-23 < 2^-12, and 63.5 is never passed from below), but for Y = 127 j: those rows are decided exactly.
struct RowScale {
  float step;    // 127 / m; of an fp32 row to 2^-21
  float limit;   // of an fp32 row quotients nearer than 0.5 - limit to a half are decided exactly; -1: every element of the row
  float pre, a;  // 2^-e, and m 2^-e: from 1 up to 2, less where m is subnormal
  float inv;     // 127 / a to 2^-21
  float most;    // m
  int ok;        // finite
  // m / 127, correctly rounded; only the thread that writes it pays for the division
  __device__ __forceinline__ float scale() const { return ok ? most / 127.f : __uint_as_float(0x7fc00000u); }
};

// B16: of 16-bit values, with m as fp32
template <bool B16>
__device__ __forceinline__ RowScale row_scale(uint32_t most) {
  RowScale s;
  s.ok = most < 0x7f800000u;
  s.most = __uint_as_float(most);
  const uint32_t e = most >> 23 ? most >> 23 : 1;
  s.pre = __uint_as_float(e >= 254 ? 0x00400000u : (254 - e) << 23);
  s.a = s.most * s.pre;
  s.inv = s.ok && most ? __fdividef(127.f, s.a) : 0.f;
  // where 127 / m or its steps leave fp32's range, every quotient is decided exactly
  bool plain = s.most >= 1e-30f && s.most <= 1e30f;
  s.step = 0.f;
  if (B16) {
    plain = plain && ((most >> 13 & 0x3ff) | 0x400) % 127 != 0;
    if (plain) {
      // at or just above 127 / a: the approximation is within 8 units
      float up = __uint_as_float(__float_as_uint(s.inv) + 8);
      const float r = fmaf(-up, s.a, 127.f);  // <= 0, exact to its sign
      up = fmaf(r, s.inv * (1.f / 127.f), up);
      if (fmaf(-up, s.a, 127.f) > 0.f) up = __uint_as_float(__float_as_uint(up) + 1);
      s.step = up * s.pre;
    }
  } else if (plain) {
    s.step = s.inv * s.pre;
  }
  s.limit = plain || most == 0 ? 0.4999f : -1.f;
  return s;
}

// q of one element, exactly: whether 127 x is above or below a half-integer times m, by products whose rounding errors are
// kept (two fused multiply-adds; near a half the rounded products are within a factor of two, so that their difference is exact).
__device__ __forceinline__ float quantize_exact(float x, const RowScale& s) {
  const float v = x * s.pre;
  const float lo = floorf(v * s.inv), half = lo + 0.5f;
  const float p = v * 127.f, pe = fmaf(v, 127.f, -p), h = half * s.a, he = fmaf(half, s.a, -h);
  const float over = (p - h) + (pe - he);
  const bool up = over > 0.f || (over == 0.f && ((int)lo & 1));
  return up ? lo + 1.f : lo;
}

constexpr float kRoundMagic = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer, halves to even

// Eight neighbouring elements -> eight bytes.
template <bool B16>
__device__ __forceinline__ uint2 quantize8(const float (&x)[8], const RowScale& s) {
  if (!s.ok) return make_uint2(0, 0);
  float t[8], off = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    t[i] = fmaf(x[i], s.step, kRoundMagic);
    if (!B16) off = fmaxf(off, fabsf(fmaf(x[i], s.step, kRoundMagic - t[i])));
  }
  if (off > s.limit) {
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = quantize_exact(x[i], s) + kRoundMagic;
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
__device__ __forceinline__ float int8_scaled(float sum, float both, float bias) {
  return __fadd_rn(__fmul_rn(sum, both), bias);
}

// ... for any scales.  Where their product leaves fp32's normal range the sum meets the smaller one first: a normal scale makes
// an integer's product no smaller than it is itself, a subnormal one makes it normal or an exact multiple of the smallest
// step, and infinite it is only where the value is.  So there are three roundings, or one to a subnormal value.
// (By selections: the branch that they replace cost a cluster's call of 64 tokens of 4096 x 4096 0.2 us.)
__device__ __forceinline__ float int8_value(int sum, float x_scale, float w_scale, float bias) {
  const float both = __fmul_rn(x_scale, w_scale);
  const bool plain = ((__float_as_uint(both) >> 23) + 1 & 0xff) >= 2;  // neither zero, subnormal, infinite nor NaN
  const bool x_first = fabsf(x_scale) < fabsf(w_scale);
  const float first = plain ? both : x_first ? x_scale : w_scale, then = plain ? 1.f : x_first ? w_scale : x_scale;
  return int8_scaled(__fmul_rn((float)sum, first), then, bias);
}

// The least and the largest size of a warp's scales that are neither 0 nor infinite nor NaN, for which any order does.
struct ScaleRange {
  uint32_t least = 0x7f800000u, most = 0;
  __device__ __forceinline__ void add(float s) {
    const uint32_t b = __float_as_uint(s) & 0x7fffffffu;
    if (b > 0 && b < 0x7f800000u) {
      least = min(least, b);
      most = max(most, b);
    }
  }
  __device__ __forceinline__ void join() {
    least = __reduce_min_sync(0xffffffffu, least);
    most = __reduce_max_sync(0xffffffffu, most);
  }
  // whether a product with w may not be normal
  __device__ __forceinline__ bool odd(float w) const {
    const float a = fabsf(w);
    if (!(a > 0.f && a <= 3.402823466e38f) || most == 0) return false;
    return __fmul_rn(__uint_as_float(least), a) < 1.17549435e-38f || __fmul_rn(__uint_as_float(most), a) > 3.402823466e38f;
  }
};

}  // namespace sesg
