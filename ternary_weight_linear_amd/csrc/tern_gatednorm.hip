// tern_gatednorm.hip -- gfx950 kernels of tern_rmsnorm_gated and
// tern_rmsnorm_post: the norms around a recurrent block, each in one pass with
// the gate, the residual's scaled addition and the int8 codes of its output.
//
// Bound by HBM (7 bytes an element: bf16 x, fp32 z, int8 codes; 13 with fp32 x
// and residual). One workgroup a token, 16 elements a thread as in the plain
// norm, everything read once and kept in registers between the reductions.
//
// Measured: gated, 2048 x 10240 to codes in 34.4 us, 4.3 TB/s; 509 x 5120 in
// groups of a head, 6.4 us. Behind a block, 2048 x 5120 to codes in 31.2 us, 4.4 TB/s; 17
// tokens 5.1 us, three trips to memory and two reductions. Copies reach 5.0 TB/s.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tern_recurrent.h"

namespace tern {
namespace {
using namespace dev;

// Chunk c of a row: two runs of 8 elements, 32 apart (16 consecutive bytes of q
// in operand order) or next to each other.
struct Chunk {
  int lo, hi;
  __device__ __forceinline__ Chunk(int c, bool apart)
      : lo(apart ? (c >> 2) * 64 + (c & 3) * 8 : c * 16), hi(lo + (apart ? 32 : 8)) {}
};

__device__ __forceinline__ void load8_of(const void* p, int64_t at, int type, float (&o)[8]) {
  if (type == TERN_F32)
    load8<TERN_F32>(p, at, o);
  else
    load8<TERN_BF16>(p, at, o);
}

// Codes of a chunk's values to row q of int8.
__device__ __forceinline__ void store_codes(const Coder& coder, const float (&v)[16], int8_t* q, int c, const Chunk& k,
                                            bool operand) {
  uint32_t w[4];
  coder.sixteen(v, w);
  if (operand) {
    *(u32x4*)(q + c * 16) = operand_order(w[0], w[1], w[2], w[3]);
  } else {
    *(uint2*)(q + k.lo) = uint2{w[0], w[1]};
    *(uint2*)(q + k.hi) = uint2{w[2], w[3]};
  }
}

__device__ __forceinline__ void store_bf16(const float (&v)[16], float factor, uint16_t* y, const Chunk& k) {
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = pack_bf16(v[8 * half + 2 * i] * factor, v[8 * half + 2 * i + 1] * factor);
    *(u32x4*)(y + (half ? k.hi : k.lo)) = o;
  }
}

// 1 / sqrt(ss / n + eps); 0 where nothing is left to divide by.
__device__ __forceinline__ float inverse_root(float ss, int n, float eps) {
  return ss == 0.f && eps == 0.f ? 0.f : 1.0f / sqrtf(ss / (float)n + eps);
}

constexpr int kMaxChunks = kNormMaxK / 16;
constexpr int kFewChunks = 8;  // a thread adds up so many of its group's sums by itself

template <int XT, int ZT, int NU>
__global__ void __launch_bounds__(1024) tern_rmsnorm_gated_kernel(GatedNormArgs a) {
  __shared__ float sums[kMaxChunks];
  __shared__ uint32_t wmax[16];
  const int64_t t = blockIdx.x;
  const int nchunk = a.K >> 4, per = a.group >> 4;  // chunks of a row, of a group
  const bool apart = a.group % 64 == 0;
  const int wave = threadIdx.x >> 6, nw = blockDim.x >> 6;
  float v[NU][16];
#pragma unroll
  for (int u = 0; u < NU; ++u) {
    const int c = threadIdx.x + blockDim.x * u;
    if (c < nchunk) {
      const Chunk k(c, apart);
      float ss = 0.f;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int at = half ? k.hi : k.lo;
        float x[8], z[8], w[8];
        load8<XT>(a.x, t * a.x_stride + at, x);
        load8<ZT>(a.z, t * a.z_stride + at, z);
        load8_of(a.w, at, a.w_type, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float g = silu(z[i]), h = a.gate_first ? x[i] * g : x[i];
          ss = __builtin_fmaf(h, h, ss);
          v[u][8 * half + i] = a.gate_first ? h * w[i] : h * w[i] * g;
        }
      }
      sums[c] = ss;
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[u][i] = 0.f;
    }
  }
  __syncthreads();
  if (per > kFewChunks) {  // one wave adds up a group, and leaves its factor at the group's first sum
    for (int g = wave; g < nchunk / per; g += nw) {
      float ss = 0.f;
      for (int c = threadIdx.x & 63; c < per; c += 64) ss += sums[g * per + c];
      ss = wave_sum(ss);
      if ((threadIdx.x & 63) == 0) sums[g * per] = inverse_root(ss, a.group, a.eps);
    }
    __syncthreads();
  }
  uint32_t m = 0;
#pragma unroll
  for (int u = 0; u < NU; ++u) {
    const int c = threadIdx.x + blockDim.x * u;
    if (c >= nchunk) break;
    const int first = c / per * per;
    float rho = sums[first];
    if (per <= kFewChunks) {
      for (int i = 1; i < per; ++i) rho += sums[first + i];
      rho = inverse_root(rho, a.group, a.eps);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      v[u][i] *= rho;
      m = max(m, __float_as_uint(v[u][i]) & 0x7fffffffu);
    }
  }
  float sc = 0.f;
  if (a.q) {
    m = wave_max_u32(m);
    if ((threadIdx.x & 63) == 0) wmax[wave] = m;
    __syncthreads();
    m = wmax[0];
    for (int w = 1; w < nw; ++w) m = max(m, wmax[w]);
    sc = __uint_as_float(m) / 127.0f;
    if (threadIdx.x == 0) a.act_scale[t] = sc;
  }
  const Coder coder(sc);
#pragma unroll
  for (int u = 0; u < NU; ++u) {
    const int c = threadIdx.x + blockDim.x * u;
    if (c >= nchunk) break;
    const Chunk k(c, apart);
    if (a.q) store_codes(coder, v[u], a.q + t * a.K, c, k, a.operand_order);
    if (a.y) store_bf16(v[u], 1.f, a.y + t * a.y_stride, k);
  }
}

// Sum and maximum over the workgroup, the same in every thread and in a fixed order.
struct Reduced {
  float sum;
  uint32_t max;
};
__device__ __forceinline__ Reduced over_workgroup(float s, uint32_t m, float* wsum, uint32_t* wmax) {
  s = wave_sum(s);
  m = wave_max_u32(m);
  if ((threadIdx.x & 63) == 0) wsum[threadIdx.x >> 6] = s, wmax[threadIdx.x >> 6] = m;
  __syncthreads();
  s = wsum[0], m = wmax[0];
  for (unsigned w = 1; w < blockDim.x >> 6; ++w) s += wsum[w], m = max(m, wmax[w]);
  return Reduced{s, m};
}

template <int XT, int RT, int NU>
__global__ void __launch_bounds__(1024) tern_rmsnorm_post_kernel(PostNormArgs a) {
  __shared__ float wsum[2][16];
  __shared__ uint32_t wmax[2][16];
  const int64_t t = blockIdx.x;
  const int nchunk = a.K >> 4;
  const bool apart = a.K % 64 == 0;
  float v[NU][16], r[NU][16];
  float ss = 0.f;
#pragma unroll
  for (int u = 0; u < NU; ++u) {
    const int c = threadIdx.x + blockDim.x * u;
#pragma unroll
    for (int i = 0; i < 16; ++i) v[u][i] = r[u][i] = 0.f;
    if (c < nchunk) {
      const Chunk k(c, apart);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int at = half ? k.hi : k.lo;
        float x[8], h[8];
        load8<XT>(a.x, t * a.x_stride + at, x);
        load8<RT>(a.r, t * a.r_stride + at, h);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[u][8 * half + i] = x[i], r[u][8 * half + i] = h[i];
          ss = __builtin_fmaf(x[i], x[i], ss);
        }
      }
    }
  }
  const float post = inverse_root(over_workgroup(ss, 0, wsum[0], wmax[0]).sum, a.K, a.eps);
  ss = 0.f;
  uint32_t m = 0;
#pragma unroll
  for (int u = 0; u < NU; ++u) {
    const int c = threadIdx.x + blockDim.x * u;
    if (c >= nchunk) break;
    const Chunk k(c, apart);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int at = half ? k.hi : k.lo;
      float pw[8], g[8], h[8];
      load8_of(a.post_w, at, a.w_type, pw);
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = 1.f;
      if (a.gate) load8_of(a.gate, t * a.gate_stride + at, a.gate_type, g);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        h[i] = r[u][8 * half + i] + a.scale * g[i] * (v[u][8 * half + i] * pw[i] * post);
      if constexpr (RT == TERN_F32) {
        f32x4* o = (f32x4*)((float*)a.r_out + t * a.r_out_stride + at);
        o[0] = f32x4{h[0], h[1], h[2], h[3]};
        o[1] = f32x4{h[4], h[5], h[6], h[7]};
      } else {
        u32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          o[i] = pack_bf16(h[2 * i], h[2 * i + 1]);
          h[2 * i] = bf16_lo(o[i]), h[2 * i + 1] = bf16_hi(o[i]);  // the norm is that of the stored stream
        }
        *(u32x4*)((uint16_t*)a.r_out + t * a.r_out_stride + at) = o;
      }
      if (a.w) {
        float w[8];
        load8_of(a.w, at, a.w_type, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          ss = __builtin_fmaf(h[i], h[i], ss);
          const float x = h[i] * w[i];
          v[u][8 * half + i] = x;
          m = max(m, __float_as_uint(x) & 0x7fffffffu);
        }
      }
    }
  }
  if (!a.w) return;  // the same in every thread
  const Reduced all = over_workgroup(ss, m, wsum[1], wmax[1]);
  // As in the plain norm: rho cancels in the quotient that is rounded, the
  // codes come from h w and its maximum alone.
  const float rho = all.max == 0 ? 0.f : 1.0f / sqrtf(all.sum / (float)a.K + a.eps);
  const float sc = __uint_as_float(all.max) / 127.0f;
  if (threadIdx.x == 0 && a.q) a.act_scale[t] = rho * sc;
  const Coder coder(sc);
#pragma unroll
  for (int u = 0; u < NU; ++u) {
    const int c = threadIdx.x + blockDim.x * u;
    if (c >= nchunk) break;
    const Chunk k(c, apart);
    if (a.q) store_codes(coder, v[u], a.q + t * a.K, c, k, a.operand_order);
    if (a.y) store_bf16(v[u], rho, a.y + t * a.y_stride, k);
  }
}

// Threads of a workgroup for rows of K, and whether each takes one chunk or two.
int threads_for(int K, bool* two) {
  const int chunks = K >> 4, nu = chunks > 1024 ? 2 : 1;
  *two = nu == 2;
  return ((chunks + nu - 1) / nu + 63) / 64 * 64;
}

template <int XT, int ZT>
void go_gated(const GatedNormArgs& a, hipStream_t st) {
  bool two;
  const int nt = threads_for(a.K, &two);
  if (two)
    tern_rmsnorm_gated_kernel<XT, ZT, 2><<<dim3(a.T), dim3(nt), 0, st>>>(a);
  else
    tern_rmsnorm_gated_kernel<XT, ZT, 1><<<dim3(a.T), dim3(nt), 0, st>>>(a);
}

template <int XT, int RT>
void go_post(const PostNormArgs& a, hipStream_t st) {
  bool two;
  const int nt = threads_for(a.K, &two);
  if (two)
    tern_rmsnorm_post_kernel<XT, RT, 2><<<dim3(a.T), dim3(nt), 0, st>>>(a);
  else
    tern_rmsnorm_post_kernel<XT, RT, 1><<<dim3(a.T), dim3(nt), 0, st>>>(a);
}

}  // namespace

int launch_rmsnorm_gated(const GatedNormArgs& a, void* stream) {
  hipStream_t st = (hipStream_t)stream;
  if (a.x_type == TERN_F32)
    a.z_type == TERN_F32 ? go_gated<TERN_F32, TERN_F32>(a, st) : go_gated<TERN_F32, TERN_BF16>(a, st);
  else
    a.z_type == TERN_F32 ? go_gated<TERN_BF16, TERN_F32>(a, st) : go_gated<TERN_BF16, TERN_BF16>(a, st);
  return kernel_launched((int)hipGetLastError(), TERN_KERNEL_RMSNORM_GATED);
}

int launch_rmsnorm_post(const PostNormArgs& a, void* stream) {
  hipStream_t st = (hipStream_t)stream;
  if (a.x_type == TERN_F32)
    a.r_type == TERN_F32 ? go_post<TERN_F32, TERN_F32>(a, st) : go_post<TERN_F32, TERN_BF16>(a, st);
  else
    a.r_type == TERN_F32 ? go_post<TERN_BF16, TERN_F32>(a, st) : go_post<TERN_BF16, TERN_BF16>(a, st);
  return kernel_launched((int)hipGetLastError(), TERN_KERNEL_RMSNORM_POST);
}

}  // namespace tern
