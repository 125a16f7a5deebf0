// tern_recurrent.h -- device-side helpers of the recurrent block's kernels
// (convolution, scan, gated norm). Internal, not installed.
#pragma once
#include "tern_decoder.h"
#include "tern_internal.h"

namespace tern {
namespace dev {

// exp(x) to about 2 ulp: the rounding of x log2(e), which the hardware's 2^t
// alone would multiply by |x|, is put back to first order. Results below
// 2^-126 are 0, above fp32 infinite; NaN stays NaN.
__device__ __forceinline__ float exp_of(float x) {
  constexpr float kHi = 0x1.715476p+0f, kLo = 0x1.4ae0cp-26f;  // log2(e) = kHi + kLo
  const float y = x < -150.f ? -150.f : x > 88.72f ? 88.72f : x;
  const float t = y * kHi;
  const float r = __builtin_fmaf(y, kLo, __builtin_fmaf(y, kHi, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  const float v = __builtin_fmaf(e, r * 0.693147182f, e);
  return x > 88.7228317f ? __builtin_inff() : v;
}

// z / (1 + exp(-z)), to about 6 + |z| / 4 roundings: the rounding of the exponent
// -z log2(e) is put back to first order, that of the constant is not. 0 from -87.33
// down, where exp(-z) passes 2^126 and its reciprocal the normal range; the value is below
// 2^-119 there.
__device__ __forceinline__ float silu(float z) {
  constexpr float kLog2e = -0x1.715476p+0f;
  const float c = __builtin_amdgcn_fmed3f(z, -126.f, 126.f), t = c * kLog2e;
  const float e = __builtin_amdgcn_exp2f(t) * __builtin_fmaf(__builtin_fmaf(c, kLog2e, -t), 0.693147182f, 1.f);
  return z * __builtin_amdgcn_rcpf(1.f + e);
}

// log(1 + exp(v)): with u = exp(-|v|) and w = 1 + u as rounded, log(1 + u) is
// log(w) and what the rounding took, over w.
__device__ __forceinline__ float softplus(float v) {
  const float u = exp_of(-fabsf(v)), w = 1.f + u;
  const float rest = (u - (w - 1.f)) * __builtin_amdgcn_rcpf(w);
  return (v > 0.f ? v : 0.f) + __builtin_fmaf(__builtin_amdgcn_logf(w), 0.693147182f, rest);
}

// Rows of sequence s in the call, [row, row + n): n is 0 for one that is left
// out. What comes from device memory is bounded here.
struct Rows {
  int64_t row;
  int n;
};
__device__ __forceinline__ Rows rows_of(const StateBatch& b, int s) {
  const int q0 = b.begin[s], q1 = b.begin[s + 1];
  if (q0 < 0 || q1 < q0 || q1 > b.rows || q1 - q0 > b.max_q) return Rows{0, 0};
  return Rows{q0, q1 - q0};
}

}  // namespace dev
}  // namespace tern
