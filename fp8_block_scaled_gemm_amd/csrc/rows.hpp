// Element types of the row operators (expert routing, expert row layout, 8-bit integer quantizer):
// fp32, bf16 and fp16 rows, read and written in 8-element pieces and computed in fp32.
#pragma once

#include "common.hpp"

namespace dg {

typedef unsigned u32x2_t __attribute__((ext_vector_type(2)));
typedef unsigned u32x4_t __attribute__((ext_vector_type(4)));

// Values of enum dg_dtype (include/dg.h).
enum Dtype : int { kF32 = 0, kBf16 = 1, kF16 = 2 };

struct Bf16 { uint16_t bits; };

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(Bf16 v) { return __uint_as_float((uint32_t)v.bits << 16); }
__device__ __forceinline__ float widen(_Float16 v) { return (float)v; }

// Round to nearest even to the row's type.
template <class T>
__device__ __forceinline__ T narrow(float v);
template <>
__device__ __forceinline__ float narrow<float>(float v) { return v; }
template <>
__device__ __forceinline__ Bf16 narrow<Bf16>(float v) { return Bf16{(uint16_t)pack2_bf16_rne(v, 0.f)}; }
template <>
__device__ __forceinline__ _Float16 narrow<_Float16>(float v) { return (_Float16)v; }

__device__ __forceinline__ uint32_t pack2_f16(float lo, float hi) {
  typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, f16x2_t{(_Float16)lo, (_Float16)hi});
}

// Eight consecutive elements as loaded: 16 bytes (32 for fp32), 16-byte aligned.
template <class T>
struct Raw8 { u32x4_t w; };
template <>
struct Raw8<float> { u32x4_t w, w2; };

template <bool NONTEMPORAL = false, class T>
__device__ __forceinline__ Raw8<T> load8(const T* p) {
  const u32x4_t* w = reinterpret_cast<const u32x4_t*>(p);
  Raw8<T> r;
  if constexpr (NONTEMPORAL) {
    r.w = __builtin_nontemporal_load(w);
    if constexpr (sizeof(T) == 4) r.w2 = __builtin_nontemporal_load(w + 1);
  } else {
    r.w = w[0];
    if constexpr (sizeof(T) == 4) r.w2 = w[1];
  }
  return r;
}

__device__ __forceinline__ void widen8(const Raw8<float>& r, float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = __uint_as_float(r.w[i]);
    v[4 + i] = __uint_as_float(r.w2[i]);
  }
}
__device__ __forceinline__ void widen8(const Raw8<Bf16>& r, float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(r.w[i] << 16);
    v[2 * i + 1] = __uint_as_float(r.w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void widen8(const Raw8<_Float16>& r, float* v) {
  typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = r.w[i];   // a copy: the compiler casts element 0 for every element of a vector lvalue
    const f16x2_t h = __builtin_bit_cast(f16x2_t, w);
    v[2 * i] = (float)h.x;
    v[2 * i + 1] = (float)h.y;
  }
}

template <class T>
__device__ __forceinline__ Raw8<T> narrow8(const float* v) {
  Raw8<T> r;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.w[i] = __float_as_uint(v[i]);
      r.w2[i] = __float_as_uint(v[4 + i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (std::is_same_v<T, Bf16>) r.w[i] = pack2_bf16_rne(v[2 * i], v[2 * i + 1]);
      else r.w[i] = pack2_f16(v[2 * i], v[2 * i + 1]);
    }
  }
  return r;
}

template <class T>
__device__ __forceinline__ void store8(T* p, const Raw8<T>& r) {
  reinterpret_cast<u32x4_t*>(p)[0] = r.w;
  if constexpr (sizeof(T) == 4) reinterpret_cast<u32x4_t*>(p)[1] = r.w2;
}

// One lane's DPP partner under a compile-time control; lanes without one (ROWS: the rows that get one)
// read 0, which lets the compiler fold the move into an unsigned maximum.
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, ROWS, 0xf, false);
}
constexpr int kDppXor1 = 0xB1, kDppXor2 = 0x4E, kDppHalfMirror = 0x141, kDppMirror = 0x140;

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Maximum over each 8-lane group, on every lane of it.
__device__ __forceinline__ uint32_t max8_u32(uint32_t v) {
  v = umax(v, dpp_u32<kDppXor1>(v));
  v = umax(v, dpp_u32<kDppXor2>(v));
  return umax(v, dpp_u32<kDppHalfMirror>(v));
}
__device__ __forceinline__ float max8(float v) {
  v = fmaxf(v, __uint_as_float(dpp_u32<kDppXor1>(__float_as_uint(v))));
  v = fmaxf(v, __uint_as_float(dpp_u32<kDppXor2>(__float_as_uint(v))));
  return fmaxf(v, __uint_as_float(dpp_u32<kDppHalfMirror>(__float_as_uint(v))));
}
// Maximum over the wave, as a wave-uniform (scalar) value: within rows of 16 lanes, then each row's last
// lane to the next row, then lane 31 to the upper half; lane 63 ends with all of it.
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  v = max8_u32(v);
  v = umax(v, dpp_u32<kDppMirror>(v));
  v = umax(v, dpp_u32<0x142, 0xa>(v));   // row_bcast:15
  v = umax(v, dpp_u32<0x143, 0xc>(v));   // row_bcast:31
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
// Sum over the wave in a fixed order (the steps of wave_max_u32), as a wave-uniform value.
__device__ __forceinline__ float wave_sum(float v) {
  v += __uint_as_float(dpp_u32<kDppXor1>(__float_as_uint(v)));
  v += __uint_as_float(dpp_u32<kDppXor2>(__float_as_uint(v)));
  v += __uint_as_float(dpp_u32<kDppHalfMirror>(__float_as_uint(v)));
  v += __uint_as_float(dpp_u32<kDppMirror>(__float_as_uint(v)));
  v += __uint_as_float(dpp_u32<0x142, 0xa>(__float_as_uint(v)));
  v += __uint_as_float(dpp_u32<0x143, 0xc>(__float_as_uint(v)));
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}

// |x| as its bit pattern: as unsigned integers these order like the magnitudes, with a NaN above
// infinity, so a maximum over them keeps a NaN.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

constexpr float kInt8Max = 127.0f;

// Scale of a row whose largest magnitude has these bits: amax / 127 (IEEE division), 1 for an
// all-zero row, NaN or infinite where the row holds such a value.
__device__ __forceinline__ float int8_scale(uint32_t amax_bits) {
  return amax_bits == 0u ? 1.0f : __uint_as_float(amax_bits) / kInt8Max;
}
// Four codes rne(v / s) (IEEE division), saturated to [-127, 127], packed little-endian; s is the same in every
// lane of the wave.  |v| <= amax keeps a quotient there by itself unless amax / 127 is subnormal: rounded to a
// few bits it lets quotients reach 190, rounded to 0 it makes them infinite.  A quotient that is not a number
// gives code 0; where the row holds one or an infinity, its scale carries it on.  Only scales outside the
// normal numbers take the instructions for all that (65536 x 1024 bf16 33.7 us, 39.5 with them for every row).
__device__ __forceinline__ uint32_t pack4_int8(const float* v, float s) {
  const uint32_t bits = (uint32_t)__builtin_amdgcn_readfirstlane((int)__float_as_uint(s));
  uint32_t w = 0;
  if (bits - 0x00800000u < 0x7f000000u) {   // 2^-126 <= s < infinity
#pragma unroll
    for (int i = 0; i < 4; ++i) w |= ((uint32_t)(int)__builtin_rintf(v[i] / s) & 0xffu) << (8 * i);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float q = v[i] / s;
      const float c = fminf(fmaxf(__builtin_rintf(q), -kInt8Max), kInt8Max);
      w |= ((uint32_t)(int)(q == q ? c : 0.0f) & 0xffu) << (8 * i);
    }
  }
  return w;
}

}  // namespace dg
