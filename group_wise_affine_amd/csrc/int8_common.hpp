// Device helpers of the int8 operators (row quantizer, int8 product, 8-bit
// cache): symmetric codes in [-127, 127] under one fp32 scale.
#pragma once

#include "mfma_common.hpp"

namespace qmm {

typedef int int4_t __attribute__((ext_vector_type(4)));
typedef int int16v_t __attribute__((ext_vector_type(16)));

// largest magnitude of eight 16-bit floats held in four words, as its bits:
// magnitudes of one sign order like their bit patterns, and infinities and
// NaN come out above every finite value
__device__ __forceinline__ uint32_t amax_pair(uint32_t m, uint32_t w) {
  typedef uint16_t us2 __attribute__((ext_vector_type(2)));
  const us2 a = __builtin_bit_cast(us2, m), b = __builtin_bit_cast(us2, w & 0x7fff7fffu);
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(a, b));
}
__device__ __forceinline__ uint32_t amax_halves(uint32_t m) {
  const uint32_t lo = m & 0xffffu, hi = m >> 16;
  return lo > hi ? lo : hi;
}

// scale of a block whose largest magnitude has these bits: fl32(amax / 127),
// NaN when the block holds an infinity or a NaN
template <class T>
__device__ __forceinline__ float amax_scale(uint32_t bits) {
  constexpr uint32_t kInf = __is_same(T, F16) ? 0x7c00u : 0x7f80u;
  if (bits >= kInf) return __builtin_nanf("");
  return to_f32(T{}, (uint16_t)bits) / 127.0f;
}

// A scale prepared for dividing by it. inv = fl32(1/s): t = fl32(v * inv) is
// within 3 * 2^-24 * |t| of fl32(v / s), so both round to the same integer
// unless t is within 2^-20 * |t| of a half-integer; only there (and for
// scales whose reciprocal would leave the normal range) the quotient itself
// is taken. s = 0 and s = NaN give codes 0.
struct Divisor {
  float s, inv;
  bool plain;
};
__device__ __forceinline__ Divisor divisor(float s) {
  Divisor d;
  d.s = s;
  d.plain = s > 0x1p-120f && s < 0x1p120f;
  d.inv = d.plain ? 1.0f / s : 0.0f;
  return d;
}
__device__ __forceinline__ bool near_half(float t, float q) {
  return fabsf(fabsf(t - q) - 0.5f) <= 0x1p-20f * fabsf(t);
}
// N codes rint(fl32(v / s)) clamped to [-127, 127], as floats
template <int N>
__device__ __forceinline__ void divide_round(const float* v, const Divisor& d, float* q) {
  bool slow = !d.plain;
#pragma unroll
  for (int i = 0; i < N; i++) {
    const float t = v[i] * d.inv;
    q[i] = __builtin_rintf(t);
    slow |= near_half(t, q[i]);
  }
  if (slow) {
    const bool any = d.s > 0.0f;   // false for 0 and NaN
#pragma unroll
    for (int i = 0; i < N; i++) q[i] = any ? __builtin_rintf(v[i] / d.s) : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < N; i++) q[i] = fminf(fmaxf(q[i], -127.0f), 127.0f);
}

__device__ __forceinline__ void unpack8(F16, const uint4& u, float* v) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const half2_t h = __builtin_bit_cast(half2_t, w[i]);
    v[2 * i] = (float)h.x;
    v[2 * i + 1] = (float)h.y;
  }
}
__device__ __forceinline__ void unpack8(BF16, const uint4& u, float* v) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; i++) {
    v[2 * i] = __builtin_bit_cast(float, w[i] << 16);
    v[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(F16, const float* v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const half2_t h = {(_Float16)v[2 * i], (_Float16)v[2 * i + 1]};
    w[i] = __builtin_bit_cast(uint32_t, h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 pack8(BF16, const float* v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const bf162_t h = {(__bf16)v[2 * i], (__bf16)v[2 * i + 1]};
    w[i] = __builtin_bit_cast(uint32_t, h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// four integral floats in [-128, 127] -> bytes, the first in the low byte
__device__ __forceinline__ uint32_t pack_codes(float a, float b, float c, float d) {
  const uint32_t ab = __builtin_amdgcn_perm((uint32_t)(int)b, (uint32_t)(int)a, 0x0c0c0400u);
  const uint32_t cd = __builtin_amdgcn_perm((uint32_t)(int)d, (uint32_t)(int)c, 0x04000c0cu);
  return ab | cd;
}
// byte i of w as a signed code
__device__ __forceinline__ float code_f32(uint32_t w, int i) {
  return (float)((int)(w << (24 - 8 * i)) >> 24);
}

__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    const uint32_t u = (uint32_t)__shfl_xor((int)v, o);
    v = u > v ? u : v;
  }
  return v;
}

}  // namespace qmm
