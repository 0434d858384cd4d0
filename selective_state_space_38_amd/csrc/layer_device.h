// Device helpers shared by the residual layer's kernels.
#pragma once

#include "layer_internal.h"
#include "ssm_device.h"

namespace ssm {

// Vector accesses at the element's alignment: gfx950 runs in unaligned access
// mode, so a row that starts anywhere moves in whole vectors all the same.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef uint32_t u32_any __attribute__((aligned(2)));

// 8 consecutive values as stored.
template <typename T>
struct Run8 : Run<T, 8> {
  using Run<T, 8>::w;
  __device__ __forceinline__ void load(const T* p) {
    const u32x4_any* q = reinterpret_cast<const u32x4_any*>(p);
#pragma unroll
    for (int i = 0; i < Run<T, 8>::NW / 4; ++i) {
      const u32x4 v = q[i];
      w[4 * i] = v[0]; w[4 * i + 1] = v[1]; w[4 * i + 2] = v[2]; w[4 * i + 3] = v[3];
    }
  }
};

// Stores values 0 .. last (of 8) at p; all of them as vectors.
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8], int last = 7) {
  if (last < 7) {
#pragma unroll
    for (int k = 0; k < 7; ++k)
      if (k <= last) store_act(p, k, v[k]);
    return;
  }
  u32x4_any* q = reinterpret_cast<u32x4_any*>(p);
  if constexpr (sizeof(T) == 2) {
    q[0] = u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                 pack_bf16x2(v[6], v[7])};
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      q[i] = u32x4{__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                   __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3])};
  }
}

// v's exchange with the lane `ROR` places further in its row of 16.
template <int ROR>
__device__ __forceinline__ float row_ror(float v) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x120 + ROR, 0xF, 0xF, true));
}

// Sum and maximum over a row of 16 lanes, in every lane.
__device__ __forceinline__ float row16_sum(float v) {
  v += row_ror<8>(v);
  v += row_ror<4>(v);
  v += row_ror<2>(v);
  v += row_ror<1>(v);
  return v;
}
__device__ __forceinline__ float row16_max(float v) {
  v = fmaxf(v, row_ror<8>(v));
  v = fmaxf(v, row_ror<4>(v));
  v = fmaxf(v, row_ror<2>(v));
  v = fmaxf(v, row_ror<1>(v));
  return v;
}

__device__ __forceinline__ float read_lane(float v, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}

// Sum over the wave, in every lane.
__device__ __forceinline__ float wave_sum(float v) {
  v = row16_sum(v);
  return (read_lane(v, 0) + read_lane(v, 16)) + (read_lane(v, 32) + read_lane(v, 48));
}

// Values of a group on the 8-bit scale: 448 (y unit) / m by a reciprocal and one
// correction.  m's mantissa and exponent are taken apart, so nothing
// overflows and the reciprocal is of a number in [1/2, 1); 448 = 2^10 7/16 and
// the product with 7/16 is exact for a bfloat16 y where unit is 1.  The
// correction leaves the quotient within half a unit, so one on a tie between two
// 8-bit values stays there.  An infinite m takes finite values to 0.
struct Fp8Scaler {
  float mul, mant, rcp;
  int exp;
  __device__ __forceinline__ explicit Fp8Scaler(float m, float unit = 1.0f) {
    const bool inf = m == __builtin_inff();
    mul = inf ? 0.0f : 0.4375f * unit;
    m = inf ? 1.0f : m;
    mant = __builtin_amdgcn_frexp_mantf(m);
    rcp = rcp_hw(mant);
    exp = 10 - __builtin_amdgcn_frexp_expf(m);
  }
  __device__ __forceinline__ float operator()(float y) const {
    const float a = y * mul;
    const float t = a * rcp;
    return __builtin_amdgcn_ldexpf(fmaf(fmaf(-t, mant, a), rcp, t), exp);
  }
};

// Four floats rounded to e4m3 (nearest even), in the order given.
__device__ __forceinline__ uint32_t pack_fp8x4(float a, float b, float c, float d) {
  int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  v = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
  return static_cast<uint32_t>(v);
}

}  // namespace ssm
