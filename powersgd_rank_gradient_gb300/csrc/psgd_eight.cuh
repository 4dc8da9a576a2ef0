// Activations in 8 bits: blocks of 128 consecutive elements of a row share a
// scale, a power of two.
//
//   scale = the least 2^e (e >= -126) with max |x| <= M 2^e over the block's finite
//           values, M the format's largest value; 1 for a block of zeros
//   code  = x / scale rounded to the format, ties to even
//
// A power of two costs at most one bit of the range above a block's largest
// value and nothing of the significands, and x / scale and code * scale are exact:
// a code is one rounding of x, restoring to fp32 or bf16 is none, and results do not hang on
// how a division was carried out.  Infinities and NaN stay visible: e5m2 has
// codes for both, e4m3 only for NaN.
#pragma once

#include <cuda_fp8.h>

#include "psgd_ops.cuh"

namespace psgd {
namespace ops {

constexpr int kBlock8 = 128;
__host__ __device__ inline long long blocks8(long long dim) { return (dim + kBlock8 - 1) / kBlock8; }

// The exponent e of a block's scale from the bits of its largest magnitude (finite).
template <bool E5> __device__ __forceinline__ int scale_exponent(unsigned top) {
  if (top == 0) return 0;
  // M is 1.75 * 2^8 (e4m3) or 1.75 * 2^15 (e5m2)
  const int q = (int)(top >> 23) - 127 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(-126, q - (E5 ? 15 : 8));
}
__device__ __forceinline__ float power2(int e) { return __uint_as_float((unsigned)(e + 127) << 23); }

// The code of v / scale (inv = 1 / scale) where v may be infinite or NaN.
template <bool E5> __device__ __forceinline__ unsigned char code_any(float v, float inv) {
  const unsigned bits = __float_as_uint(v), sign = (bits >> 24) & 0x80u, mag = bits & 0x7fffffffu;
  if (mag > 0x7f800000u || (!E5 && mag == 0x7f800000u)) return (unsigned char)(sign | 0x7fu);
  if (mag == 0x7f800000u) return (unsigned char)(sign | 0x7cu);
  return (unsigned char)__nv_cvt_float_to_fp8(v * inv, __NV_SATFINITE, E5 ? __NV_E5M2 : __NV_E4M3);
}
// Two finite values' codes, the first in the low byte.
template <bool E5> __device__ __forceinline__ unsigned codes2(float x, float y) {
  return __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, E5 ? __NV_E5M2 : __NV_E4M3);
}
// What two codes in the low bits stand for, without their scale.
template <bool E5> __device__ __forceinline__ float2 values2(unsigned c) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)c, E5 ? __NV_E5M2 : __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Largest magnitude's bits over the LANES neighbouring lanes that share a block.
template <int LANES> __device__ __forceinline__ unsigned lanes_max(unsigned m) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

// Codes of a block's N values (N = 4 or 8) of this lane, packed from the low byte on, and the block's scale, where
// something in the block is infinite or NaN: the scale is that of the others.  All of the block's LANES lanes are here,
// of a warp's other block perhaps none, so the lanes are named.
template <int N, int LANES, bool E5>
__device__ __forceinline__ void encode_special(const float (&v)[N], unsigned (&packed)[N / 4], float& scale) {
  unsigned top = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const unsigned m = __float_as_uint(v[i]) & 0x7fffffffu;
    if (m < 0x7f800000u) top = max(top, m);
  }
  const unsigned mask = LANES == 32 ? 0xffffffffu : ((1u << (LANES & 31)) - 1u) << (threadIdx.x & 31 & ~(LANES - 1));
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(mask, top, o));
  const int e = scale_exponent<E5>(top);
  const float inv = power2(-e);
  scale = power2(e);
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    packed[i] = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) packed[i] |= (unsigned)code_any<E5>(v[4 * i + k], inv) << (8 * k);
  }
}

// The same where all is finite, or perhaps not.
template <int N, int LANES, bool E5>
__device__ __forceinline__ void encode(const float (&v)[N], unsigned (&packed)[N / 4], float& scale) {
  unsigned all = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) all = max(all, __float_as_uint(v[i]) & 0x7fffffffu);
  all = lanes_max<LANES>(all);
  if (all >= 0x7f800000u) {
    encode_special<N, LANES, E5>(v, packed, scale);
    return;
  }
  const int e = scale_exponent<E5>(all);
  const float inv = power2(-e);
  scale = power2(e);
#pragma unroll
  for (int i = 0; i < N / 4; ++i)
    packed[i] = codes2<E5>(v[4 * i] * inv, v[4 * i + 1] * inv) | codes2<E5>(v[4 * i + 2] * inv, v[4 * i + 3] * inv) << 16;
}
template <int N, int LANES>
__device__ __forceinline__ void encode(bool e5, const float (&v)[N], unsigned (&packed)[N / 4], float& scale) {
  if (e5) encode<N, LANES, true>(v, packed, scale);
  else encode<N, LANES, false>(v, packed, scale);
}

// Four codes times their scale.
__device__ __forceinline__ void decode4(bool e5, unsigned packed, float scale, float* f) {
  const float2 a = e5 ? values2<true>(packed & 0xffffu) : values2<false>(packed & 0xffffu);
  const float2 b = e5 ? values2<true>(packed >> 16) : values2<false>(packed >> 16);
  f[0] = a.x * scale;
  f[1] = a.y * scale;
  f[2] = b.x * scale;
  f[3] = b.y * scale;
}
__device__ __forceinline__ float decode1(bool e5, unsigned char c, float scale) {
  return (e5 ? values2<true>(c).x : values2<false>(c).x) * scale;
}

}  // namespace ops
}  // namespace psgd
