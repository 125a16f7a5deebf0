// tern_conv.hip -- gfx950 kernel of tern_causal_conv: the short causal
// convolution in front of the scan, with its state.
//
//   y[t][c] = act(bias[c] + sum_i w[c][i] x[t - (W - 1) + i][c]),  W = 2..4.
//
// Bound by HBM: 6 bytes an element with fp32 input. A thread takes 16 bytes of
// channels and a run of tokens, whose window of W - 1 earlier rows stays in
// registers, so a row is read once, and W - 1 rows twice at the runs' ends.
// The thread of a sequence's first run reads the old state before it writes
// the new one, and no other thread reads that slot.
//
// Measured (W = 4): 2048 tokens of 12288 channels, fp32, in 30.6 us, 4.9 TB/s, the rate of
// a copy; runs of 8 tokens take 55 us, of 32 30.0. 32 single tokens, bf16, in 5.5 us, two
// trips to memory and a launch.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tern_recurrent.h"

namespace tern {
namespace {
using namespace dev;

constexpr int kRun = 16;  // tokens a thread
constexpr int kStep = 8;  // rows asked for together

template <int TYPE>
constexpr int kChannels = TYPE == TERN_F32 ? 4 : 8;  // 16 bytes

template <int TYPE>
__device__ __forceinline__ void widen(const u32x4& w, float (&o)[kChannels<TYPE>]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (TYPE == TERN_F32)
      o[i] = __uint_as_float(w[i]);
    else
      o[2 * i] = bf16_lo(w[i]), o[2 * i + 1] = bf16_hi(w[i]);
  }
}

// N consecutive weights (N a multiple of 4) of either type.
template <int N>
__device__ __forceinline__ void load_weights(const void* p, int64_t at, int type, float (&o)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    if (type == TERN_F32) {
      const f32x4 v = *(const f32x4*)((const float*)p + at + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i + j] = v[j];
    } else {
      const uint2 v = *(const uint2*)((const uint16_t*)p + at + i);
      o[i] = bf16_lo(v.x), o[i + 1] = bf16_hi(v.x), o[i + 2] = bf16_lo(v.y), o[i + 3] = bf16_hi(v.y);
    }
  }
}

template <int TYPE, int W>
__global__ void __launch_bounds__(256) tern_causal_conv_kernel(ConvArgs a) {
  constexpr int CH = kChannels<TYPE>, BYTES = 16 / CH;
  const int s = blockIdx.y;
  const int blocks = a.channels / CH;
  const int at = blockIdx.x * 256 + threadIdx.x;  // below 2^31, which the host sees to
  const int run = at / blocks, c0 = (at - run * blocks) * CH;
  const int t0 = run * kRun;
  // What does not depend on the batch's arrays is asked for before them: a single
  // token waits for two trips to memory, one for the arrays and one for the rest.
  float w[CH * W], bias[CH];
  load_weights(a.w, (int64_t)c0 * W, a.w_type, w);
#pragma unroll
  for (int i = 0; i < CH; ++i) bias[i] = 0.f;
  if (a.bias) load_weights(a.bias, c0, a.w_type, bias);
  const int src = a.batch.src[s], dst = a.batch.dst[s];
  const Rows r = rows_of(a.batch, s);
  if (t0 >= r.n) return;
  const char* x = (const char*)a.x + (r.row * a.x_stride + c0) * BYTES;
  const int64_t step = a.x_stride * BYTES;
  const int last = min(t0 + kRun, r.n);
  u32x4 raw[kStep], old[W - 1];
#pragma unroll
  for (int j = 0; j < kStep; ++j)
    if (t0 + j < last) raw[j] = *(const u32x4*)(x + (t0 + j) * step);
  const int64_t slot = (int64_t)(W - 1) * a.channels;  // elements
  if (run > 0) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) old[j] = *(const u32x4*)(x + (t0 - (W - 1) + j) * step);
  } else {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      old[j] = u32x4{0, 0, 0, 0};
      if (src >= 0 && src < a.slots)
        old[j] = *(const u32x4*)((const char*)a.state + (src * slot + (int64_t)j * a.channels + c0) * BYTES);
    }
  }
  float past[W - 1][CH];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) widen<TYPE>(old[j], past[j]);
  uint16_t* y = a.y + r.row * a.y_stride + c0;
  for (int t = t0;;) {
#pragma unroll
    for (int j = 0; j < kStep; ++j) {
      if (t + j >= last) break;
      float now[CH], o[CH];
      widen<TYPE>(raw[j], now);
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        float v = bias[i];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) v = __builtin_fmaf(w[i * W + k], past[k][i], v);
        v = __builtin_fmaf(w[i * W + W - 1], now[i], v);
        o[i] = a.silu ? silu(v) : v;
#pragma unroll
        for (int k = 0; k + 1 < W - 1; ++k) past[k][i] = past[k + 1][i];
        past[W - 2][i] = now[i];
      }
      uint32_t out[CH / 2];
#pragma unroll
      for (int i = 0; i < CH / 2; ++i) out[i] = pack_bf16(o[2 * i], o[2 * i + 1]);
      if constexpr (CH == 4)
        *(uint2*)(y + (t + j) * a.y_stride) = uint2{out[0], out[1]};
      else
        *(u32x4*)(y + (t + j) * a.y_stride) = u32x4{out[0], out[1], out[2], out[3]};
    }
    if ((t += kStep) >= last) break;
#pragma unroll
    for (int j = 0; j < kStep; ++j)
      if (t + j < last) raw[j] = *(const u32x4*)(x + (t + j) * step);
  }
  if (run == 0 && dst >= 0 && dst < a.slots) {
    // new state j: input n - (W - 1) + j of this call, or from the old state before it
    u32x4 now[W - 1];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      const int i = r.n - (W - 1) + j;
      now[j] = old[W - 2];
#pragma unroll
      for (int o = 0; o < W - 1; ++o)
        if (i == o - (W - 1)) now[j] = old[o];
      if (i >= 0) now[j] = *(const u32x4*)(x + i * step);
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
      *(u32x4*)((char*)a.state + (dst * slot + (int64_t)j * a.channels + c0) * BYTES) = now[j];
  }
}

template <int TYPE>
void go(const ConvArgs& a, dim3 grid, hipStream_t st) {
  if (a.width == 2)
    tern_causal_conv_kernel<TYPE, 2><<<grid, dim3(256), 0, st>>>(a);
  else if (a.width == 3)
    tern_causal_conv_kernel<TYPE, 3><<<grid, dim3(256), 0, st>>>(a);
  else
    tern_causal_conv_kernel<TYPE, 4><<<grid, dim3(256), 0, st>>>(a);
}

int64_t blocks_of_sequence(const ConvArgs& a) {
  const int64_t threads = (int64_t)(a.channels / (a.type == TERN_F32 ? 4 : 8)) * ((a.batch.max_q + kRun - 1) / kRun);
  return (threads + 255) / 256;
}

}  // namespace

int64_t conv_blocks(const ConvArgs& a) { return blocks_of_sequence(a) * a.batch.seqs; }

int launch_conv(const ConvArgs& a, void* stream) {
  const dim3 grid((unsigned)blocks_of_sequence(a), a.batch.seqs);
  if (a.type == TERN_F32)
    go<TERN_F32>(a, grid, (hipStream_t)stream);
  else
    go<TERN_BF16>(a, grid, (hipStream_t)stream);
  return kernel_launched((int)hipGetLastError(), TERN_KERNEL_CAUSAL_CONV);
}

}  // namespace tern
