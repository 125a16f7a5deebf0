// tern_norm.hip -- gfx950 kernel of tern_rmsnorm: the residual's addition, the
// RMS norm and the per-token int8 quantisation of its output in one pass.
//
//   h = x + r (fp32), rounded to the residual's type and stored;
//   v = h w;  rho = 1 / sqrt(sum h^2 / K + eps);
//   y = v rho (bf16);  q = clamp(rne(v / (max|v| / 127))),  scale = rho max|v| / 127.
//
// rho is one positive factor per token, so it cancels in the quotient that is
// rounded: the codes come from v and its maximum alone and do not depend on
// the rounding of the sum of squares. Both reductions therefore run together
// (one barrier), and every element is read once and kept in registers.
//
// Bound by HBM: 13 bytes an element with fp32 input and residual. One
// workgroup a token with 16 elements a thread (K = 5120: 5 waves, 24 VGPRs)
// keeps enough tokens in flight: 2048 x 5120 takes 27.4 us = 4.97 TB/s, the
// rate of a plain device copy (5.1 TB/s); 509 x 5120 in bf16 7.5 us; one token
// 3.5 us, which is the launch and one trip to memory.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tern_decoder.h"
#include "tern_internal.h"

namespace tern {
namespace {
using namespace dev;

// One workgroup per token; each thread owns up to NU chunks of 16 elements in
// two runs of 8: 32 apart, which makes 16 consecutive bytes of q in operand
// order, or next to each other where K is no multiple of 64. The layout of q
// does not enter, so both layouts give the same scales to the last bit. RT:
// the residual's type, or -1 for none.
template <int XT, int RT, int NU>
__global__ void __launch_bounds__(1024) tern_rmsnorm_kernel(NormArgs a) {
  __shared__ float wsum[16];
  __shared__ uint32_t wmax[16];
  const int64_t t = blockIdx.x;
  const int nchunk = a.K >> 4;
  const bool apart = a.K % 64 == 0;
  float v[NU][16];
  float ss = 0.f;
  uint32_t m = 0;
#pragma unroll
  for (int u = 0; u < NU; ++u) {
    const int c = threadIdx.x + blockDim.x * u;
    if (c < nchunk) {
      const int lo = apart ? (c >> 2) * 64 + (c & 3) * 8 : c * 16;
      const int hi = lo + (apart ? 32 : 8);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int k = half ? hi : lo;
        float h[8], w[8];
        load8<XT>(a.x, t * a.x_stride + k, h);
        if constexpr (RT >= 0) {
          float r[8];
          load8<RT>(a.r, t * a.r_stride + k, r);
#pragma unroll
          for (int i = 0; i < 8; ++i) h[i] += r[i];
          if constexpr (RT == TERN_F32) {
            f32x4* o = (f32x4*)((float*)a.r_out + t * a.r_out_stride + k);
            o[0] = f32x4{h[0], h[1], h[2], h[3]};
            o[1] = f32x4{h[4], h[5], h[6], h[7]};
          } else {
            u32x4 o;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              o[i] = pack_bf16(h[2 * i], h[2 * i + 1]);
              h[2 * i] = bf16_lo(o[i]), h[2 * i + 1] = bf16_hi(o[i]);  // the norm is that of the stored stream
            }
            *(u32x4*)((uint16_t*)a.r_out + t * a.r_out_stride + k) = o;
          }
        }
        if (a.w_type == TERN_F32)
          load8<TERN_F32>(a.w, k, w);
        else
          load8<TERN_BF16>(a.w, k, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          ss = __builtin_fmaf(h[i], h[i], ss);
          const float x = h[i] * w[i];
          v[u][8 * half + i] = x;
          m = max(m, __float_as_uint(x) & 0x7fffffffu);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[u][i] = 0.f;
    }
  }
  ss = wave_sum(ss);
  m = wave_max_u32(m);
  const int nw = blockDim.x >> 6;
  if ((threadIdx.x & 63) == 0) wsum[threadIdx.x >> 6] = ss, wmax[threadIdx.x >> 6] = m;
  __syncthreads();
  ss = wsum[0], m = wmax[0];
  for (int w = 1; w < nw; ++w) ss += wsum[w], m = max(m, wmax[w]);
  // Without an eps rho is infinite for a token of zeros, and y would be 0 * inf.
  const float rho = m == 0 ? 0.f : 1.0f / sqrtf(ss / (float)a.K + a.eps);
  const float sc = __uint_as_float(m) / 127.0f;
  if (threadIdx.x == 0 && a.q) a.act_scale[t] = rho * sc;
  const Coder coder(sc);
#pragma unroll
  for (int u = 0; u < NU; ++u) {
    const int c = threadIdx.x + blockDim.x * u;
    if (c >= nchunk) break;
    const int lo = apart ? (c >> 2) * 64 + (c & 3) * 8 : c * 16;
    const int hi = lo + (apart ? 32 : 8);
    if (a.q) {
      uint32_t w[4];
      coder.sixteen(v[u], w);
      if (a.operand_order) {
        *(u32x4*)(a.q + t * a.K + c * 16) = operand_order(w[0], w[1], w[2], w[3]);
      } else {
        *(uint2*)(a.q + t * a.K + lo) = uint2{w[0], w[1]};
        *(uint2*)(a.q + t * a.K + hi) = uint2{w[2], w[3]};
      }
    }
    if (a.y) {
      uint16_t* y = a.y + t * a.y_stride;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        u32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = pack_bf16(v[u][8 * half + 2 * i] * rho, v[u][8 * half + 2 * i + 1] * rho);
        *(u32x4*)(y + (half ? hi : lo)) = o;
      }
    }
  }
}

template <int XT, int RT>
void go(const NormArgs& a, hipStream_t st) {
  const int chunks = a.K >> 4;
  const int nu = chunks > 1024 ? 2 : 1;
  const int nt = ((chunks + nu - 1) / nu + 63) / 64 * 64;
  if (nu == 1)
    tern_rmsnorm_kernel<XT, RT, 1><<<dim3(a.T), dim3(nt), 0, st>>>(a);
  else
    tern_rmsnorm_kernel<XT, RT, 2><<<dim3(a.T), dim3(nt), 0, st>>>(a);
}

template <int XT>
void go_x(const NormArgs& a, hipStream_t st) {
  if (a.r_type < 0)
    go<XT, -1>(a, st);
  else if (a.r_type == TERN_F32)
    go<XT, TERN_F32>(a, st);
  else
    go<XT, TERN_BF16>(a, st);
}

}  // namespace

int launch_rmsnorm(const NormArgs& a, void* stream) {
  hipStream_t st = (hipStream_t)stream;
  if (a.x_type == TERN_F32)
    go_x<TERN_F32>(a, st);
  else
    go_x<TERN_BF16>(a, st);
  return kernel_launched((int)hipGetLastError(), TERN_KERNEL_RMSNORM);
}

}  // namespace tern
