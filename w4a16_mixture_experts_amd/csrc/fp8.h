// 8-bit values with scales: e4m3 (4 exponent bits, 3 of the fraction, largest 448, no infinities),
// one fp32 scale per 128 neighbours. A value is q * scale with
//   scale = max(largest |v| of the 128 / 448, 2^-126),   q = e4m3(v / scale), to nearest even.
// A group that holds a NaN gets a NaN scale. All of it is IEEE arithmetic on 32-bit values: with an
// infinity the scale is infinite, so the group's finite values are 0 x inf = NaN, as by the formula.
// v / scale is formed as v * (1 / scale): one division per group, off by at most 1.5 units in the
// last of 24 bits before it is rounded to 4.
#pragma once

#include <type_traits>

#include "common.h"
#include "device.h"

namespace exmoe {

typedef float f32x8 __attribute__((ext_vector_type(8)));

// Eight elements off, off + 1, .. of an array of any alignment (a global access of 8 or 16 bytes
// may start at any address on this device), the first n of them where n < 8: the others are zeros and
// not touched.
template <int DT>
struct Elems;
template <>
struct Elems<EXMOE_DTYPE_FP32> {
  typedef float type;
  static constexpr int kBytes = 4;
  typedef float f32x4_u __attribute__((ext_vector_type(4), aligned(4)));
  static __device__ __forceinline__ float get(const void* p, size_t i) { return static_cast<const float*>(p)[i]; }
  static __device__ __forceinline__ void put(void* p, size_t i, float v) { static_cast<float*>(p)[i] = v; }
  static __device__ __forceinline__ float rounded(float v) { return v; }
  static __device__ __forceinline__ f32x8 load8(const void* p, size_t off) {
    const f32x4_u* q = reinterpret_cast<const f32x4_u*>(static_cast<const float*>(p) + off);
    const f32x4_u a = q[0], b = q[1];
    return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  }
  static __device__ __forceinline__ f32x4 load4(const void* p, size_t off) {
    return *reinterpret_cast<const f32x4_u*>(static_cast<const float*>(p) + off);
  }
  static __device__ __forceinline__ void store4(void* p, size_t off, f32x4 v) {
    *reinterpret_cast<f32x4_u*>(static_cast<float*>(p) + off) = v;
  }
  static __device__ __forceinline__ void store8(void* p, size_t off, f32x8 v) {
    f32x4_u* q = reinterpret_cast<f32x4_u*>(static_cast<float*>(p) + off);
    q[0] = f32x4_u{v[0], v[1], v[2], v[3]};
    q[1] = f32x4_u{v[4], v[5], v[6], v[7]};
  }
};
// 16-bit types: F the conversion of one value each way
template <class F>
struct Elems16 {
  typedef uint16_t type;
  static constexpr int kBytes = 2;
  typedef uint32_t u32x4_u __attribute__((ext_vector_type(4), aligned(2)));
  static __device__ __forceinline__ float get(const void* p, size_t i) { return F::to_f32(static_cast<const uint16_t*>(p)[i]); }
  static __device__ __forceinline__ void put(void* p, size_t i, float v) { static_cast<uint16_t*>(p)[i] = F::from_f32(v); }
  static __device__ __forceinline__ float rounded(float v) { return F::to_f32(F::from_f32(v)); }
  static __device__ __forceinline__ f32x8 load8(const void* p, size_t off) {
    const u32x4_u w = *reinterpret_cast<const u32x4_u*>(static_cast<const uint16_t*>(p) + off);
    f32x8 v;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      v[2 * i] = F::to_f32((uint16_t)w[i]);
      v[2 * i + 1] = F::to_f32((uint16_t)(w[i] >> 16));
    }
    return v;
  }
  typedef uint32_t u32x2_u __attribute__((ext_vector_type(2), aligned(2)));
  static __device__ __forceinline__ f32x4 load4(const void* p, size_t off) {
    const u32x2_u w = *reinterpret_cast<const u32x2_u*>(static_cast<const uint16_t*>(p) + off);
    return f32x4{F::to_f32((uint16_t)w[0]), F::to_f32((uint16_t)(w[0] >> 16)), F::to_f32((uint16_t)w[1]), F::to_f32((uint16_t)(w[1] >> 16))};
  }
  static __device__ __forceinline__ void store4(void* p, size_t off, f32x4 v) {
    *reinterpret_cast<u32x2_u*>(static_cast<uint16_t*>(p) + off) = u32x2_u{F::pack2(v[0], v[1]), F::pack2(v[2], v[3])};
  }
  static __device__ __forceinline__ void store8(void* p, size_t off, f32x8 v) {
    u32x4_u w;
#pragma unroll
    for (int i = 0; i < 4; i++) w[i] = F::pack2(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<u32x4_u*>(static_cast<uint16_t*>(p) + off) = w;
  }
};
struct ConvBF16 {
  static __device__ __forceinline__ float to_f32(uint16_t v) { return bf16_to_f32(v); }
  static __device__ __forceinline__ uint16_t from_f32(float v) { return f32_to_bf16(v); }
  static __device__ __forceinline__ uint32_t pack2(float lo, float hi) { return pack_bf16x2(lo, hi); }
};
struct ConvFP16 {
  static __device__ __forceinline__ float to_f32(uint16_t v) { return (float)__builtin_bit_cast(_Float16, v); }
  static __device__ __forceinline__ uint16_t from_f32(float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }
  static __device__ __forceinline__ uint32_t pack2(float lo, float hi) { return (uint32_t)from_f32(lo) | ((uint32_t)from_f32(hi) << 16); }
};
template <>
struct Elems<EXMOE_DTYPE_BF16> : Elems16<ConvBF16> {};
template <>
struct Elems<EXMOE_DTYPE_FP16> : Elems16<ConvFP16> {};

template <int DT>
__device__ __forceinline__ f32x8 load_upto8(const void* p, size_t off, int n) {
  if (n >= 8) return Elems<DT>::load8(p, off);
  f32x8 v = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 7; i++)
    if (i < n) v[i] = Elems<DT>::get(p, off + i);
  return v;
}
template <int DT>
__device__ __forceinline__ void store_upto8(void* p, size_t off, int n, f32x8 v) {
  if (n >= 8) {
    Elems<DT>::store8(p, off, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < 7; i++)
    if (i < n) Elems<DT>::put(p, off + i, v[i]);
}

constexpr float kF8Most = 448.f;
constexpr float kF8LeastScale = 0x1p-126f;

// Largest |v| as its bit pattern, whose order is that of the magnitudes, NaN above all of them.
__device__ __forceinline__ uint32_t abs_bits8(f32x8 v) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; i++) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return m;
}
// ... of the 16 lanes of a row, in each of them
__device__ __forceinline__ uint32_t row16_max_u32(uint32_t v) {
  v = max(v, dpp_u32<0x121>(v));   // row_ror:1
  v = max(v, dpp_u32<0x122>(v));
  v = max(v, dpp_u32<0x124>(v));
  v = max(v, dpp_u32<0x128>(v));
  return v;
}
__device__ __forceinline__ float f8_scale(uint32_t abs_bits) {
  const float s = __uint_as_float(abs_bits) / kF8Most;
  return s < kF8LeastScale ? kF8LeastScale : s;   // (false for NaN)
}
// e4m3 of eight values times inv = 1 / scale (the hardware's conversion rounds to nearest even;
// values over 448 (1 + 1/28) would become NaN, and none is)
__device__ __forceinline__ uint2 f8_pack8(f32x8 v, float inv) {
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * inv, v[1] * inv, 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2] * inv, v[3] * inv, lo, true);
  int hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4] * inv, v[5] * inv, 0, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6] * inv, v[7] * inv, hi, true);
  return make_uint2((uint32_t)lo, (uint32_t)hi);
}
__device__ __forceinline__ void f8_store(uint8_t* p, int n, uint2 q) {
  typedef uint32_t u32x2_u __attribute__((ext_vector_type(2), aligned(1)));
  if (n >= 8) {
    *reinterpret_cast<u32x2_u*>(p) = u32x2_u{q.x, q.y};
    return;
  }
#pragma unroll
  for (int i = 0; i < 7; i++)
    if (i < n) p[i] = (uint8_t)((i < 4 ? q.x : q.y) >> (8 * (i & 3)));
}

// Calls f with the type as a constant.
template <class F>
inline hipError_t by_dtype(int dtype, F f) {
  if (dtype == EXMOE_DTYPE_BF16) return f(std::integral_constant<int, EXMOE_DTYPE_BF16>{});
  if (dtype == EXMOE_DTYPE_FP16) return f(std::integral_constant<int, EXMOE_DTYPE_FP16>{});
  return f(std::integral_constant<int, EXMOE_DTYPE_FP32>{});
}
inline int dtype_bytes(int dtype) { return dtype == EXMOE_DTYPE_FP32 ? 4 : 2; }

}  // namespace exmoe
