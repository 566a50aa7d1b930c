// Arithmetic shared by the layer operators' kernels: 16-bit conversions,
// activations and their derivatives, and the 8-bit block format.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>
#include <type_traits>

#include "layer.h"

namespace dion3 {
namespace lm {

// --------------------------------------------------------------------------
// Elements
// --------------------------------------------------------------------------
template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// Two values packed into one 32-bit word of 16-bit elements, and back.
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (BF16) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&t);
  } else {
    const __half2 t = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&t);
  }
}
template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (BF16)
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  else
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <bool BF16>
__device__ __forceinline__ uint16_t pack1(float a) {
  if constexpr (BF16)
    return __bfloat16_as_ushort(__float2bfloat16_rn(a));
  else
    return __half_as_ushort(__float2half_rn(a));
}
template <bool BF16>
__device__ __forceinline__ float unpack1(uint16_t h) {
  if constexpr (BF16)
    return __uint_as_float(static_cast<uint32_t>(h) << 16);
  else
    return __half2float(__ushort_as_half(h));
}

// VEC contiguous elements as fp32; VEC = 8 needs 16-byte aligned addresses.
template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T* p, float (&v)[VEC]) {
  if constexpr (VEC == 8 && sizeof(T) == 2) {
    constexpr bool kBf = sizeof(T) == 2 && std::is_same<T, __nv_bfloat16>::value;
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack2<kBf>(w[i]);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  } else if constexpr (VEC == 8) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    static_assert(VEC == 1, "one element or eight");
    v[0] = to_f32<T>(*p);
  }
}
template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T* p, const float (&v)[VEC]) {
  if constexpr (VEC == 8 && sizeof(T) == 2) {
    constexpr bool kBf = std::is_same<T, __nv_bfloat16>::value;
    *reinterpret_cast<uint4*>(p) = make_uint4(pack2<kBf>(v[0], v[1]), pack2<kBf>(v[2], v[3]),
                                              pack2<kBf>(v[4], v[5]), pack2<kBf>(v[6], v[7]));
  } else if constexpr (VEC == 8) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *p = from_f32<T>(v[0]);
  }
}

// --------------------------------------------------------------------------
// Activations.  gelu is its tanh form, 0.5 z (1 + tanh(sqrt(2/pi) (z + c z^3)))
// = z / (1 + exp(-2 sqrt(2/pi) (z + c z^3))), c = 0.044715: written with the
// sigmoid it does not cancel at large -z.  The sigmoid takes two special
// function instructions, 2^x and 1/x (each within 2 ulp; results below 2^-126
// become 0), and the slope's cubic term is bounded where the sigmoid's own
// slope is 0, so derivatives stay finite for every finite z.
// --------------------------------------------------------------------------
constexpr float kGelu2 = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kLog2E = 1.4426950408889634f;

__device__ __forceinline__ float sigmoid(float u) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-kLog2E * u));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return r;
}
__device__ __forceinline__ float gelu_arg(float z) { return z * fmaf(0.044715f * kGelu2, z * z, kGelu2); }

template <int ACT>
__device__ __forceinline__ float act_fwd(float z) {
  if constexpr (ACT == kActNone) return z;
  if constexpr (ACT == kActRelu) return z > 0.f ? z : (z != z ? z : 0.f);
  if constexpr (ACT == kActGelu) return z * sigmoid(gelu_arg(z));
  return z * sigmoid(z);
}
template <int ACT>
__device__ __forceinline__ float act_grad(float z) {
  if constexpr (ACT == kActNone) return 1.f;
  if constexpr (ACT == kActRelu) return z > 0.f ? 1.f : (z != z ? z : 0.f);
  if constexpr (ACT == kActGelu) {
    const float s = sigmoid(gelu_arg(z)), zd = z * fmaf(-s, s, s);
    return fmaf(zd, kGelu2 * fmaf(0.134145f, fminf(z * z, 1e9f), 1.f), s);
  }
  const float s = sigmoid(z);
  return fmaf(z, fmaf(-s, s, s), s);
}

// --------------------------------------------------------------------------
// 8-bit blocks.  A block's scale is 2^e with e the smallest integer in
// [-127, 121] such that amax <= 127 2^e; the byte is e + 127.  127 = 1.984375 *
// 2^6, so with amax = 1.m 2^E the exponent is E - 6, one more if 1.m >
// 1.984375 (mantissa bits > 0x7E0000).  Magnitudes above 127 2^121 = 3.376e38
// saturate there: the next scale would round them to 2^128.  Byte 255: some
// value was NaN or infinite, and the block stands for NaN.  Codes are v 2^-e
// rounded to the nearest integer (ties to even), at most 127 in magnitude, so
// a value q 2^e has 7 significant bits: exact in bf16 and fp32 and, within its
// range, in fp16.
// --------------------------------------------------------------------------
constexpr uint32_t kTopByte = 248u;

__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
  const int e = static_cast<int>(amax_bits >> 23);
  if (e == 255) return 255u;
  const int b = e - 6 + ((amax_bits & 0x7FFFFFu) > 0x7E0000u ? 1 : 0);
  return min(static_cast<uint32_t>(b > 0 ? b : 0), kTopByte);
}
__device__ __forceinline__ float inv_scale(uint32_t byte) {  // 2^-e; 0 for byte 255
  return byte == 255u ? 0.f : __uint_as_float((254u - byte) << 23);
}
__device__ __forceinline__ float scale_of(uint32_t byte) {  // 2^e; NaN for byte 255
  return byte == 255u ? __uint_as_float(0x7FC00000u) : byte == 0u ? __uint_as_float(0x00400000u)
                                                                  : __uint_as_float(byte << 23);
}
// Values of a block as they are coded: saturated in the one scale where that
// can matter.
template <int N>
__device__ __forceinline__ void saturate_block(uint32_t byte, float (&v)[N]) {
  if (byte == kTopByte) {
    constexpr float kMost = 127.f * 2658455991569831745807614120560689152.f;  // 127 2^121
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = fminf(fmaxf(v[j], -kMost), kMost);
  }
}
// Code of v as the low 8 bits: v * inv is exact up to underflow, and adding
// 1.5 * 2^23 rounds it to an integer held in the low mantissa bits.  `inv` is
// 0 when the block stands for NaN; the code is then 0 too (the select keeps
// NaN and infinity times 0 out of it).
__device__ __forceinline__ uint32_t code_of(float v, float inv) {
  const float f = fmaf(v, inv, 12582912.f);
  return inv == 0.f ? 0u : (__float_as_uint(f) & 0xFFu);
}
// Four codes in one word.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float inv) {
  const uint32_t x = __float_as_uint(fmaf(a, inv, 12582912.f)), y = __float_as_uint(fmaf(b, inv, 12582912.f));
  const uint32_t z = __float_as_uint(fmaf(c, inv, 12582912.f)), w = __float_as_uint(fmaf(d, inv, 12582912.f));
  const uint32_t r = __byte_perm(__byte_perm(x, y, 0x0040), __byte_perm(z, w, 0x0040), 0x5410);
  return inv == 0.f ? 0u : r;
}
// The values of four codes: 2^23 + (q + 128) is built from the code's bits and
// the 2^23 + 128 taken off again, both exact.
__device__ __forceinline__ void values4(uint32_t w, float scale, float (&v)[4]) {
  const uint32_t u = w ^ 0x80808080u;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    v[j] = (__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440 + j)) - 8388736.f) * scale;
}
// Larger magnitude of two values; NaN if either is.
__device__ __forceinline__ float max_mag(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}

// The same for two packed 16-bit values each.
template <bool BF16>
__device__ __forceinline__ uint32_t max_mag2(uint32_t a, uint32_t b) {
  if constexpr (BF16) {
    const __nv_bfloat162 r = __hmax2_nan(__habs2(*reinterpret_cast<const __nv_bfloat162*>(&a)),
                                         __habs2(*reinterpret_cast<const __nv_bfloat162*>(&b)));
    return *reinterpret_cast<const uint32_t*>(&r);
  } else {
    const __half2 r = __hmax2_nan(__habs2(*reinterpret_cast<const __half2*>(&a)),
                                  __habs2(*reinterpret_cast<const __half2*>(&b)));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
}

}  // namespace lm
}  // namespace dion3
