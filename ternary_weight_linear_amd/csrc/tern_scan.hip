// tern_scan.hip -- gfx950 kernel of tern_scan for few rows a sequence: the
// selective state space scan token by token.
//
//   S[t] = exp(D[t] a) S[t-1] + D[t] B[t] x[t]^T  (N x P),  y[t] = C[t] S[t] + d x[t].
//
// tern_scan_step_kernel goes token by token with the state in registers. Bound
// by HBM: 8 N P bytes of state a head and call against 5 N P operations a
// token. A workgroup takes one sequence and head; lane l of a wave holds 4 of
// the P columns (16 bytes of a state row) of N / 4 / (256 / P) rows, so C S is summed in
// the lane and crosses lanes once a token.
//
// Measured (160 heads of 64 x 128): one token of 32 sequences 65 us, 5.2 TB/s of
// states read and written, as a copy; 4 tokens of 16 sequences 39 us, 4.3 TB/s (each
// further token costs about 2 us, its reduction and barrier); one token of one sequence
// 4.9 us, the launch and three trips to memory.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tern_recurrent.h"

namespace tern {
namespace {
using namespace dev;

// R consecutive bf16 as they lie in memory.
template <int R>
struct Raw {
  uint32_t w[R / 2];
  __device__ __forceinline__ void load(const uint16_t* p) {
    if constexpr (R == 2) {
      w[0] = *(const uint32_t*)p;
    } else if constexpr (R == 4) {
      const uint2 v = *(const uint2*)p;
      w[0] = v.x, w[1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < R / 8; ++i) {
        const u32x4 v = ((const u32x4*)p)[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[4 * i + j] = v[j];
      }
    }
  }
  __device__ __forceinline__ float at(int i) const { return i & 1 ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]); }
};

__device__ __forceinline__ float load_dt(const ScanArgs& a, int64_t row, int h) {
  const int64_t at = row * a.dt_stride + h;
  return a.dt_type == TERN_F32 ? ((const float*)a.dt)[at] : __uint_as_float((uint32_t)((const uint16_t*)a.dt)[at] << 16);
}

// Sums over lanes 32 apart of a (in the lower lanes) and b (in the upper ones).
__device__ __forceinline__ float halves(float a, float b) {
  const auto v = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  return __uint_as_float(v[0]) + __uint_as_float(v[1]);
}
// Sums over lanes 16 apart of a (in rows 0 and 2 of 16 lanes) and b (in rows 1 and 3).
__device__ __forceinline__ float rows16(float a, float b) {
  const auto v = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  return __uint_as_float(v[0]) + __uint_as_float(v[1]);
}

template <int P, int N>
__global__ void __launch_bounds__(256) tern_scan_step_kernel(ScanArgs a) {
  constexpr int LPR = P / 4, NG = 64 / LPR, R = N / 4 / NG;
  __shared__ float part[2][4][P];
  const int s = blockIdx.x / a.heads, h = blockIdx.x - s * a.heads;
  const Rows r = rows_of(a.batch, s);
  if (r.n == 0) return;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int p4 = lane % LPR * 4, n0 = wave * (N / 4) + lane / LPR * R;
  const int64_t head = (int64_t)h * N * P, slot = (int64_t)a.heads * N * P;
  const int at = n0 * P + p4;
  f32x4 st[R];
  const int src = a.batch.src[s];
  if (src >= 0 && src < a.slots) {
    const float* from = a.state + src * slot + head + at;
#pragma unroll
    for (int i = 0; i < R; ++i) st[i] = *(const f32x4*)(from + i * P);
  } else {
#pragma unroll
    for (int i = 0; i < R; ++i) st[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  const int g = h / (a.heads / a.groups);
  const uint16_t* x = a.x + r.row * a.x_stride + h * P + p4;
  const uint16_t* b = a.b + r.row * a.b_stride + g * N + n0;
  const uint16_t* c = a.c + r.row * a.c_stride + g * N + n0;
  const int upper = lane >> 5, mine = (lane >> 4 & 1) * 2 + upper;  // columns that the lane ends
  const float decay = a.a[h], bias = a.dt_bias ? a.dt_bias[h] : 0.f, skip = a.d ? a.d[h] : 0.f;
  Raw<4> xt;
  Raw<R> bt, ct;
  xt.load(x), bt.load(b), ct.load(c);
  float dt = load_dt(a, r.row, h);
  for (int t = 0; t < r.n; ++t) {
    const Raw<4> xn = xt;
    const Raw<R> bn = bt, cn = ct;
    float D = dt + bias;
    if (t + 1 < r.n) {
      xt.load(x + (t + 1) * a.x_stride), bt.load(b + (t + 1) * a.b_stride), ct.load(c + (t + 1) * a.c_stride);
      dt = load_dt(a, r.row + t + 1, h);
    }
    if (a.softplus) D = softplus(D);
    const float keep = exp_of(D * decay);
    float u[4], y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = D * xn.at(i), y[i] = 0.f;
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const float bk = bn.at(k), ck = cn.at(k);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        st[k][i] = __builtin_fmaf(bk, u[i], keep * st[k][i]);
        y[i] = __builtin_fmaf(ck, st[k][i], y[i]);
      }
    }
    if (a.d && threadIdx.x < LPR) {
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = __builtin_fmaf(skip, xn.at(i), y[i]);
    }
    // The lanes that hold the same columns add up, each ending one or two of the four.
    float* to = part[t & 1][wave] + p4;
    if constexpr (P == 128) {
      to[upper] = halves(y[0], y[1]), to[2 + upper] = halves(y[2], y[3]);
    } else {
      float v = rows16(halves(y[0], y[1]), halves(y[2], y[3]));
      if constexpr (P == 32) v += __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), 0x128, 0xf, 0xf, true));  // row_ror:8
      if (lane % 16 < LPR) to[mine] = v;
    }
    __syncthreads();  // the other half of `part` was read before the barrier of the token in between
    if (threadIdx.x < P / 2) {
      const int p = threadIdx.x * 2;
      float o[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const auto& v = part[t & 1];
        o[i] = (v[0][p + i] + v[1][p + i]) + (v[2][p + i] + v[3][p + i]);
      }
      *(uint32_t*)(a.y + ((r.row + t) * a.heads + h) * P + p) = pack_bf16(o[0], o[1]);
    }
  }
  const int dst = a.batch.dst[s];
  if (dst >= 0 && dst < a.slots) {
    float* to = a.state + dst * slot + head + at;
#pragma unroll
    for (int i = 0; i < R; ++i) *(f32x4*)(to + i * P) = st[i];
  }
}

template <int P>
void go_step(const ScanArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)(a.batch.seqs * a.heads));
  if (a.state_dim == 64)
    tern_scan_step_kernel<P, 64><<<grid, dim3(256), 0, st>>>(a);
  else if (a.state_dim == 128)
    tern_scan_step_kernel<P, 128><<<grid, dim3(256), 0, st>>>(a);
  else
    tern_scan_step_kernel<P, 256><<<grid, dim3(256), 0, st>>>(a);
}

}  // namespace

int launch_scan_step(const ScanArgs& a, void* stream) {
  hipStream_t st = (hipStream_t)stream;
  if (a.dim == 32)
    go_step<32>(a, st);
  else if (a.dim == 64)
    go_step<64>(a, st);
  else
    go_step<128>(a, st);
  return kernel_launched((int)hipGetLastError(), TERN_KERNEL_SCAN_STEP);
}

}  // namespace tern
