// Shared device helpers of the row operators over the vocabulary (vocab_adjust.cu,
// vocab_top.cu, vocab_distill.cu): base-2 sums of exponentials and ordered keys.
#pragma once

#include "common.cuh"

namespace dory {

// The hardware's approximation, within 2^-22 of the value (fp32 rounds to 2^-24);
// results below 2^-126 are 0.  In a softmax that is far below an fp32 share's use,
// and a kernel that takes every logit's exponential twice has no issue slots for a
// longer form.
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

// Running sum of exponentials: s = sum of 2^(c (x - m)) over the values taken
// so far, m their maximum.  x - m is formed first: it is exact next to the
// maximum, and further off its rounding is relative to the difference, whereas
// a rounded c m would scale the whole sum by up to an ulp of |c m|.
// Empty, or every value -inf: m = -inf, s = 0.  A NaN value makes s NaN;
// without one, +inf makes it +inf (m = +inf).
struct ExpSum {
  float m, s;
};
// what to subtract in exponents: the maximum, 0 while there is none, and a finite
// value below +inf, so that only a NaN gives NaN
__device__ __forceinline__ float exp_ref(float m) {
  return m == -INFINITY ? 0.f : fminf(m, 3.402823466e38f);
}
// a softmax's sum: infinite values have no shares, NaN
__device__ __forceinline__ ExpSum softmax_sum(ExpSum a) { return {a.m, a.m == INFINITY ? NAN : a.s}; }

__device__ __forceinline__ float exp_term(float x, float c, float ref) {
  return exp2_fast((x - ref) * c);
}
// make room for values up to `top` (their maximum): call before adding them
__device__ __forceinline__ void exp_raise(ExpSum& a, float top, float c) {
  if (top > a.m) {
    a.s *= exp_term(a.m, c, top);
    a.m = top;
  }
}
__device__ __forceinline__ ExpSum exp_join(ExpSum a, ExpSum b, float c) {
  const float m = fmaxf(a.m, b.m), ref = exp_ref(m);
  return {m, a.s * exp_term(a.m, c, ref) + b.s * exp_term(b.m, c, ref)};
}
// 2^(c (x - ref)) for many x, in one fused multiply-add each: 2^(c x - d) with
// d = c ref rounded, and `fix` = 2^(d - c ref) the factor that its rounding
// left out.  For |d| < 1024 the rounding is below 2^-14, where 1 - log(2) r has
// an error of r^2 / 4 < 2^-30.  Beyond, the difference comes first as above.
struct ExpBase {
  float ref, d, fix;
  bool near;
};
__device__ __forceinline__ ExpBase exp_base(float m, float c) {
  ExpBase b;
  b.ref = exp_ref(m);
  b.d = b.ref * c;
  b.near = fabsf(b.d) < 1024.f;
  b.fix = b.near ? fmaf(-0.69314718f, fmaf(b.ref, c, -b.d), 1.f) : 1.f;
  return b;
}
// two fp32 operations in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)),
        "l"(reinterpret_cast<uint64_t&>(c)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return d;
}
template <bool kNear>
__device__ __forceinline__ float4 exp4_at(const float4& x, float c, const ExpBase& b) {
  float2 u, v;
  if (kNear) {
    const float2 cc = make_float2(c, c), dd = make_float2(-b.d, -b.d);
    u = fma2(make_float2(x.x, x.y), cc, dd);
    v = fma2(make_float2(x.z, x.w), cc, dd);
  } else {
    u = make_float2((x.x - b.ref) * c, (x.y - b.ref) * c);
    v = make_float2((x.z - b.ref) * c, (x.w - b.ref) * c);
  }
  return make_float4(exp2_fast(u.x), exp2_fast(u.y), exp2_fast(v.x), exp2_fast(v.y));
}
template <bool kNear, int N>
__device__ __forceinline__ float exp_sum_at(const float4 (&x)[N], float c, const ExpBase& b) {
  float2 s = make_float2(0.f, 0.f), t = s;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float4 e = exp4_at<kNear>(x[i], c, b);
    s = add2(s, make_float2(e.x, e.y));
    t = add2(t, make_float2(e.z, e.w));
  }
  s = add2(s, t);
  return s.x + s.y;
}
__device__ __forceinline__ float max4(const float4& x) { return fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w)); }
// add N float4 to a running sum
template <int N>
__device__ __forceinline__ void exp_add(ExpSum& a, const float4 (&x)[N], float c) {
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < N; ++i) top = fmaxf(top, max4(x[i]));
  exp_raise(a, top, c);
  const ExpBase b = exp_base(a.m, c);
  a.s += (b.near ? exp_sum_at<true>(x, c, b) : exp_sum_at<false>(x, c, b)) * b.fix;
}

// over the 32 lanes: the maximum first, then one rescaling each
__device__ __forceinline__ ExpSum warp_join(ExpSum a, float c) {
  const float m = warp_max(a.m);
  return {m, warp_sum(a.s * exp_term(a.m, c, exp_ref(m)))};
}

// Order-preserving key of a float: a < b iff key(a) < key(b), -0 and +0 equal,
// every NaN key 0 (below -inf).
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0u;
  const uint32_t b = __float_as_uint(x + 0.f);
  return b ^ ((b & 0x80000000u) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  if (k == 0u) return __uint_as_float(0x7FFFFFFFu);
  return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}

}  // namespace dory
