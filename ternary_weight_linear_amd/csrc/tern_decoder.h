// tern_decoder.h -- device-side helpers of the decoder operators' kernels
// (norm, cache, attention). Internal, not installed.
#pragma once
#include <type_traits>

#include "tern_device.h"

namespace tern {
namespace dev {

// ---- int8 codes: clamp(rne(fl(v / scale)), -127, 127), the rule of the s8
// rung's quantisation, for scales that many values share.
struct Coder {
  float scale, inv;
  bool by_inv;  // the scale is a normal float, so its reciprocal is finite

  __device__ __forceinline__ explicit Coder(float s) : scale(s), inv(1.0f / s), by_inv(s >= 0x1p-126f) {}
  static __device__ __forceinline__ uint32_t byte(float r) { return (uint32_t)(int)fminf(fmaxf(r, -127.f), 127.f) & 0xffu; }
  // By division: IEEE quotient, ties to even; a NaN becomes -127, a zero scale gives 0.
  __device__ __forceinline__ uint32_t divided(float v) const { return scale == 0.f ? 0u : byte(rintf(v / scale)); }
  // By the reciprocal, or `near` is set: for |v| <= 127 scale the product lies
  // within 2^-16 of v / scale and the IEEE quotient within 2^-17, so unless it
  // is within 2^-15 of a half-integer both round to the same integer.
  __device__ __forceinline__ uint32_t quick(float v, bool& near) const {
    const float y = v * inv, t = rintf(y);
    near |= !(by_inv && fabsf(y - t) < 0.5f - 0x1p-15f);
    return byte(t);
  }
  __device__ __forceinline__ uint32_t one(float v) const {
    bool near = false;
    const uint32_t c = quick(v, near);
    return near ? divided(v) : c;
  }
  // 16 codes, byte e of dword d that of value 4 d + e.
  __device__ __forceinline__ void sixteen(const float (&v)[16], uint32_t (&w)[4]) const {
    bool near = false;
#pragma unroll
    for (int d = 0; d < 4; ++d)
      w[d] = quick(v[4 * d], near) | quick(v[4 * d + 1], near) << 8 | quick(v[4 * d + 2], near) << 16 |
             quick(v[4 * d + 3], near) << 24;
    if (near) {
#pragma unroll
      for (int d = 0; d < 4; ++d)
        w[d] = divided(v[4 * d]) | divided(v[4 * d + 1]) << 8 | divided(v[4 * d + 2]) << 16 |
               divided(v[4 * d + 3]) << 24;
    }
  }
};

// The s8 contraction's byte order inside a 64-wide block (TERN_Q_OPERAND_ORDER):
// 16 bytes from the codes of elements 8g..8g+7 (L0, L1) and 32+8g.. (H0, H1).
__device__ __forceinline__ u32x4 operand_order(uint32_t L0, uint32_t L1, uint32_t H0, uint32_t H1) {
  return u32x4{__builtin_amdgcn_perm(H0, L0, 0x01050004u), __builtin_amdgcn_perm(H0, L0, 0x03070206u),
               __builtin_amdgcn_perm(H1, L1, 0x01050004u), __builtin_amdgcn_perm(H1, L1, 0x03070206u)};
}

// ---- bf16 conversions and reductions.

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// Two floats rounded to nearest even bf16, packed (NaN stays NaN).
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 v = {(__bf16)lo, (__bf16)hi};
  return __builtin_bit_cast(uint32_t, v);
}

// Sum over the 64 lanes, the same in every lane and in a fixed order: a
// butterfly inside each row of 16 lanes (every lane of a pair adds the same
// two numbers), then the four row sums.
__device__ __forceinline__ float wave_sum(float v) {
  auto dpp = [](float x, auto ctrl) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(x), decltype(ctrl)::value, 0xf,
                                                                 0xf, false));
  };
  v += dpp(v, std::integral_constant<int, 0xb1>{});   // quad_perm [1,0,3,2]
  v += dpp(v, std::integral_constant<int, 0x4e>{});   // quad_perm [2,3,0,1]
  v += dpp(v, std::integral_constant<int, 0x141>{});  // row_half_mirror
  v += dpp(v, std::integral_constant<int, 0x140>{});  // row_mirror
  auto lane = [&](int i) { return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), i)); };
  return (lane(0) + lane(16)) + (lane(32) + lane(48));
}
}  // namespace dev
}  // namespace tern
