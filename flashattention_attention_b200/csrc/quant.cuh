// quant.cuh -- element loads and the int8 row quantiser's arithmetic, shared by
// the quantiser and one-token append (quant.cu) and the rotated paged append
// (rope_append.cu), whose int8 codes must agree bit for bit.  quant.cu
// explains the arithmetic.
#pragma once

#include "device.cuh"

namespace fa {

// Raw vector loads of 4 consecutive elements (kept raw in registers while
// the next rows are in flight) and their exact widening to fp32.
template <typename T>
struct Vec4;
template <>
struct Vec4<float> {
  using Raw = float4;
  __device__ __forceinline__ static Raw load(const float* p) { return __ldcs(reinterpret_cast<const float4*>(p)); }
  __device__ __forceinline__ static Raw zero() { return make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ static void widen(const Raw& t, float (&v)[4]) {
    v[0] = t.x; v[1] = t.y; v[2] = t.z; v[3] = t.w;
  }
};
template <>
struct Vec4<__nv_bfloat16> {
  using Raw = uint2;
  __device__ __forceinline__ static Raw load(const __nv_bfloat16* p) {
    return __ldcs(reinterpret_cast<const uint2*>(p));
  }
  __device__ __forceinline__ static Raw zero() { return make_uint2(0u, 0u); }
  // bf16 -> fp32 is exact: the bf16 bits are the top half of the fp32 bits.
  __device__ __forceinline__ static void widen(const Raw& t, float (&v)[4]) {
    v[0] = __uint_as_float(t.x << 16);
    v[1] = __uint_as_float(t.x & 0xffff0000u);
    v[2] = __uint_as_float(t.y << 16);
    v[3] = __uint_as_float(t.y & 0xffff0000u);
  }
};

// IEEE-division path: any s (0 gives zero codes), with the clamp.
__device__ __forceinline__ uint32_t quantise4_div(const float (&v)[4], float s) {
  uint32_t packed = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    int c = 0;
    if (s > 0.0f) {
      c = __float2int_rn(__fdiv_rn(v[e], s));  // IEEE division, round half to even
      c = max(-127, min(127, c));
    }
    packed |= (static_cast<uint32_t>(c) & 0xffu) << (8 * e);
  }
  return packed;
}

// Fast path for s in [2^-60, 2^60]: y = RN(1 / s); Markstein's correction
// step gives the correctly rounded x / s, and the 1.5 * 2^23 shift rounds it
// half to even into the low byte.
__device__ __forceinline__ uint32_t quantise4_fast(const float (&v)[4], float s, float y) {
  const float2 y2 = make_float2(y, y), ns2 = make_float2(-s, -s);
  const float2 shift = make_float2(12582912.0f, 12582912.0f);  // 1.5 * 2^23
  uint32_t t[4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float2 x = make_float2(v[2 * h], v[2 * h + 1]);
    const float2 q0 = mul2(x, y2);
    const float2 r = fma2(q0, ns2, x);  // x - q0 s, exact
    const float2 q = fma2(r, y2, q0);
    const float2 k = add2(q, shift);
    t[2 * h] = __float_as_uint(k.x);
    t[2 * h + 1] = __float_as_uint(k.y);
  }
  uint32_t lo, hi, packed;
  asm("prmt.b32 %0, %1, %2, 0x0040;" : "=r"(lo) : "r"(t[0]), "r"(t[1]));
  asm("prmt.b32 %0, %1, %2, 0x0040;" : "=r"(hi) : "r"(t[2]), "r"(t[3]));
  asm("prmt.b32 %0, %1, %2, 0x5410;" : "=r"(packed) : "r"(lo), "r"(hi));
  return packed;
}

}  // namespace fa
