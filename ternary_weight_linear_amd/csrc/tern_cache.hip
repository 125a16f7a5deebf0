// tern_cache.hip -- gfx950 kernels of the 8-bit paged key/value cache: the
// append of new tokens (rotary positions of several axes on q and k, then k
// and v quantised into their pages) and the reader that gives stored values
// back as bf16.
//
// A page holds 64 tokens; a page and kv head have one scale for their keys
// and one for their values. Places inside a page and head:
//   k: byte slot * d + i                 (slot 0..63, element i)
//   v: byte i * 64 + 16 g + 4 tile + e   for slot 16 tile + 4 g + e
// so that the attention's lanes find the four 4-token runs that a matrix
// instruction's operand takes in 16 consecutive bytes.
//
// Bound by HBM for prompts, by a launch and a chain of dependent loads for
// single tokens. A workgroup takes one page, head and kind: the page's new
// values stay in registers between their maximum and their codes (64 x 128
// values: 36 VGPRs), so everything is read once; the kept part of a page is
// touched only when its scale grows. The same launch turns q. A 2048-token
// prompt with 40 + 16 heads of 128 in fp32 takes 17.9 us for 84 MB (4.7 TB/s,
// a plain device copy runs at 5.1), 32 decode tokens 5.4 us; reading the
// touched pages back 7.1 us each.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tern_decoder.h"
#include "tern_internal.h"

namespace tern {
namespace {
using namespace dev;

// What one workgroup handles: the slots [lo, hi) of one page of a sequence,
// and the row of `tokens` that slot lo comes from or goes to.
struct PageSpan {
  int64_t page;  // page id, -1: nothing to do
  int lo, hi;
  int64_t row;
  bool kept;  // slots below lo hold tokens of earlier calls
};

// Span `p` of sequence s's new tokens [kv - n, kv): page (kv - n) / 64 + p.
// Every value that comes from device memory is bounded here, so that tables
// that contradict the host's sizes cannot lead outside the buffers.
__device__ __forceinline__ PageSpan page_span(const KvBatch& b, int64_t pages, int tokens, int s, int p) {
  PageSpan r;
  r.page = -1;
  r.lo = r.hi = 0;
  r.row = 0;
  r.kept = false;
  const int q0 = b.q_begin[s], q1 = b.q_begin[s + 1];
  const int kv = b.kv_len[s];
  if (q0 < 0 || q1 < q0 || q1 > tokens || kv < 0 || kv > b.max_kv) return r;  // q1 - q0 below does not wrap
  const int n = q1 - q0;
  if (n <= 0 || n > b.max_q || n > kv) return r;
  const int start = kv - n;
  const int at = start / kKvPage + p;  // page of the sequence
  const int first = max(start, at * kKvPage), last = min(kv, (at + 1) * kKvPage);
  if (first >= last || at >= b.table_width) return r;
  const int id = b.page_table[(int64_t)s * b.table_width + at];
  if (id < 0 || id >= pages) return r;
  r.page = id;
  r.lo = first - at * kKvPage;
  r.hi = last - at * kKvPage;
  r.row = q0 + (first - start);
  r.kept = r.lo > 0;
  return r;
}

template <int TYPE>
__device__ __forceinline__ void load4(const void* p, int64_t at, float (&o)[4]) {
  if constexpr (TYPE == TERN_F32) {
    const f32x4 a = *(const f32x4*)((const float*)p + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = a[i];
  } else {
    const uint2 w = *(const uint2*)((const uint16_t*)p + at);
    o[0] = bf16_lo(w.x), o[1] = bf16_hi(w.x), o[2] = bf16_lo(w.y), o[3] = bf16_hi(w.y);
  }
}

// Elements of chunk c (0..d/8-1) of a head: two runs of 4, A and B. The
// first rot/8 chunks hold pairs (A[i], B[i]) = elements (4c + i, rot/2 + 4c + i)
// that turn together; the others lie next to each other and do not turn.
__device__ __forceinline__ void chunk_at(int c, int pairs, int& a, int& b, bool& turns) {
  turns = 4 * c < pairs;
  a = turns ? 4 * c : 8 * c;
  b = turns ? pairs + 4 * c : 8 * c + 4;
}

// Turns the four pairs of chunk c of token row `row`. Each product and sum is
// rounded by itself, as in separate elementwise operations.
__device__ __forceinline__ void turn(const RopeArgs& r, int64_t tokens, int64_t row, int c, float (&A)[4], float (&B)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int pair = 4 * c + i;
    const int axis = min((int)r.axis[pair], r.axes - 1);
    const int pos = min(max(r.positions[axis * tokens + row], 0), r.max_pos - 1);
    const float2 cs = ((const float2*)r.table)[(int64_t)pos * r.pairs + pair];
    const float x = A[i], y = B[i];
    A[i] = x * cs.x - y * cs.y;
    B[i] = y * cs.x + x * cs.y;
  }
}

// Codes of earlier calls on a page whose scale grows from `from` to `to`.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float from, float to) {
  const Coder coder(to);
  uint32_t o = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float c = (float)(int8_t)(w >> (8 * e));
    o |= coder.divided(c * from) << (8 * e);
  }
  return o;
}

constexpr int kThreads = 256;

// Maximum of `m` over the workgroup.
__device__ __forceinline__ uint32_t block_max(uint32_t m, uint32_t* lds) {
  m = wave_max_u32(m);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = m;
  __syncthreads();
  return max(max(lds[0], lds[1]), max(lds[2], lds[3]));
}

// New scale of a page: that of the new values, or the one it has if it
// already holds tokens of a larger one.
__device__ __forceinline__ float new_scale(uint32_t m, const PageSpan& p, float old) {
  const float s = __uint_as_float(m) / 127.0f;
  return p.kept && !(s > old) && s == s ? old : s;
}

// Keys of one page and head: turned, then quantised. 4 runs of codes a
// thread and token chunk stay in registers between the maximum and the codes.
template <int D, int TYPE>
__device__ __forceinline__ void append_k(const KvAppendArgs& a, const PageSpan& p, int head, uint32_t* lds) {
  constexpr int C = D / 8;                        // chunks a token
  constexpr int N = kKvPage * C / kThreads;       // chunks a thread
  const int64_t ph = p.page * a.cache.heads + head;
  int8_t* page = a.cache.k + ph * kKvPage * D;
  float* scale = a.cache.k_scale + ph;
  const float old = *scale;
  float A[N][4], B[N][4];
  uint32_t m = 0;
#pragma unroll
  for (int u = 0; u < N; ++u) {
    const int item = threadIdx.x + kThreads * u;
    const int slot = p.lo + item / C, c = item % C;
    if (slot < p.hi) {
      int ia, ib;
      bool turns;
      chunk_at(c, a.rope.pairs, ia, ib, turns);
      const int64_t row = p.row + slot - p.lo;
      const int64_t at = row * a.k_stride + (int64_t)head * D;
      load4<TYPE>(a.k, at + ia, A[u]);
      load4<TYPE>(a.k, at + ib, B[u]);
      if (turns) turn(a.rope, a.tokens, row, c, A[u], B[u]);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        m = max(m, max(__float_as_uint(A[u][i]) & 0x7fffffffu, __float_as_uint(B[u][i]) & 0x7fffffffu));
    }
  }
  m = block_max(m, lds);
  const float sc = new_scale(m, p, old);
  if (p.kept && sc != old) {  // the tokens below lo, on the new scale
    uint32_t* w = (uint32_t*)page;
    for (int i = threadIdx.x; i < p.lo * D / 4; i += kThreads) w[i] = rescale4(w[i], old, sc);
  }
  if (threadIdx.x == 0) *scale = sc;
  const Coder coder(sc);
#pragma unroll
  for (int u = 0; u < N; ++u) {
    const int item = threadIdx.x + kThreads * u;
    const int slot = p.lo + item / C, c = item % C;
    if (slot < p.hi) {
      int ia, ib;
      bool turns;
      chunk_at(c, a.rope.pairs, ia, ib, turns);
      uint32_t wa = 0, wb = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        wa |= coder.one(A[u][i]) << (8 * i);
        wb |= coder.one(B[u][i]) << (8 * i);
      }
      *(uint32_t*)(page + slot * D + ia) = wa;
      *(uint32_t*)(page + slot * D + ib) = wb;
    }
  }
}

// Values of one page and head. A thread takes 4 elements of a run of 4 slots
// (16 x D/4 such blocks a page), which are four dwords of the page.
template <int D, int TYPE>
__device__ __forceinline__ void append_v(const KvAppendArgs& a, const PageSpan& p, int head, uint32_t* lds) {
  constexpr int E = D / 4;
  constexpr int N = 16 * E / kThreads;
  const int64_t ph = p.page * a.cache.heads + head;
  int8_t* page = a.cache.v + ph * kKvPage * D;
  float* scale = a.cache.v_scale + ph;
  const float old = *scale;
  float V[N][4][4];
  uint32_t m = 0;
#pragma unroll
  for (int u = 0; u < N; ++u) {
    const int item = threadIdx.x + kThreads * u;
    const int run = p.lo / 4 + item / E, e = item % E;  // runs from the first new slot on: short spans touch few
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int slot = 4 * run + t;
      if (slot >= p.lo && slot < p.hi) {
        load4<TYPE>(a.v, (p.row + slot - p.lo) * a.v_stride + (int64_t)head * D + 4 * e, V[u][t]);
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max(m, __float_as_uint(V[u][t][i]) & 0x7fffffffu);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) V[u][t][i] = 0.f;
      }
    }
  }
  m = block_max(m, lds);
  const float sc = new_scale(m, p, old);
  if (p.kept && sc != old) {
    // Every dword of the page: slots from lo on are written below or unused.
    uint32_t* w = (uint32_t*)page;
    for (int i = threadIdx.x; i < kKvPage * D / 4; i += kThreads) w[i] = rescale4(w[i], old, sc);
    __syncthreads();  // before new codes go into the same dwords
  }
  if (threadIdx.x == 0) *scale = sc;
  const Coder coder(sc);
#pragma unroll
  for (int u = 0; u < N; ++u) {
    const int item = threadIdx.x + kThreads * u;
    const int run = p.lo / 4 + item / E, e = item % E;
    if (4 * run >= p.hi) continue;
    const int place = 16 * (run & 3) + 4 * (run >> 2);
    const bool whole = 4 * run >= p.lo && 4 * run + 4 <= p.hi;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      int8_t* d = page + (4 * e + i) * kKvPage + place;
      uint32_t c[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) c[t] = coder.one(V[u][t][i]);
      if (whole) {
        *(uint32_t*)d = c[0] | (c[1] << 8) | (c[2] << 16) | (c[3] << 24);
      } else {
#pragma unroll
        for (int t = 0; t < 4; ++t)
          if (4 * run + t >= p.lo && 4 * run + t < p.hi) d[t] = (int8_t)c[t];
      }
    }
  }
}

// Grid: `spans` x heads x 2 x seqs workgroups of keys and values, then the
// workgroups that turn q, one chunk of 8 elements a thread.
template <int D, int TYPE>
__global__ void __launch_bounds__(kThreads) tern_kv_append_kernel(KvAppendArgs a, int spans, unsigned kv_blocks) {
  __shared__ uint32_t lds[4];
  if (blockIdx.x < kv_blocks) {
    unsigned i = blockIdx.x;
    const int which = i & 1;
    i >>= 1;
    const int head = i % a.cache.heads;
    i /= a.cache.heads;
    const int span = i % spans, s = i / spans;
    const PageSpan p = page_span(a.batch, a.cache.pages, a.tokens, s, span);
    if (p.page < 0) return;
    if (which == 0)
      append_k<D, TYPE>(a, p, head, lds);
    else
      append_v<D, TYPE>(a, p, head, lds);
    return;
  }
  constexpr int C = D / 8;
  const int64_t i = (int64_t)(blockIdx.x - kv_blocks) * kThreads + threadIdx.x;
  const int c = (int)(i % C);
  const int64_t rh = i / C;
  const int64_t row = rh / a.q_heads;
  const int head = (int)(rh - row * a.q_heads);
  if (row >= a.tokens) return;
  int ia, ib;
  bool turns;
  chunk_at(c, a.rope.pairs, ia, ib, turns);
  float A[4], B[4];
  const int64_t at = row * a.q_stride + (int64_t)head * D;
  load4<TYPE>(a.q, at + ia, A);
  load4<TYPE>(a.q, at + ib, B);
  if (turns) turn(a.rope, a.tokens, row, c, A, B);
  uint16_t* o = a.q_out + rh * D;
  *(uint2*)(o + ia) = uint2{pack_bf16(A[0], A[1]), pack_bf16(A[2], A[3])};
  *(uint2*)(o + ib) = uint2{pack_bf16(B[0], B[1]), pack_bf16(B[2], B[3])};
}

// The stored values of every sequence's last tokens, as bf16 [rows][heads][d].
template <int D>
__global__ void __launch_bounds__(kThreads) tern_kv_read_kernel(KvReadArgs a, int spans) {
  unsigned i = blockIdx.x;
  const int which = i & 1;
  i >>= 1;
  const int head = i % a.cache.heads;
  i /= a.cache.heads;
  const int span = i % spans, s = i / spans;
  const PageSpan p = page_span(a.batch, a.cache.pages, a.rows, s, span);
  if (p.page < 0) return;
  const int64_t ph = p.page * a.cache.heads + head;
  uint16_t* out = (which == 0 ? a.k_out : a.v_out);
  if (!out) return;
  if (which == 0) {
    constexpr int C = D / 8;
    const int8_t* page = a.cache.k + ph * kKvPage * D;
    const float sc = a.cache.k_scale[ph];
    for (int item = threadIdx.x; item < (p.hi - p.lo) * C; item += kThreads) {
      const int t = item / C, c = item % C;
      const uint2 w = *(const uint2*)(page + (p.lo + t) * D + 8 * c);
      u32x4 o;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t x = (j < 2 ? w.x : w.y) >> (16 * (j & 1));
        o[j] = pack_bf16((float)(int8_t)x * sc, (float)(int8_t)(x >> 8) * sc);
      }
      *(u32x4*)(out + ((p.row + t) * a.cache.heads + head) * D + 8 * c) = o;
    }
  } else {
    constexpr int E = D / 4;
    const int8_t* page = a.cache.v + ph * kKvPage * D;
    const float sc = a.cache.v_scale[ph];
    for (int item = threadIdx.x; item < 16 * E; item += kThreads) {
      const int run = p.lo / 4 + item / E, e = item % E;
      if (4 * run >= p.hi) break;
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = *(const uint32_t*)(page + (4 * e + j) * kKvPage + 16 * (run & 3) + 4 * (run >> 2));
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int slot = 4 * run + t;
        if (slot < p.lo || slot >= p.hi) continue;
        float f[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = (float)(int8_t)(w[j] >> (8 * t)) * sc;
        *(uint2*)(out + ((p.row + slot - p.lo) * a.cache.heads + head) * D + 4 * e) =
            uint2{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3])};
      }
    }
  }
}

// Pages that n tokens in a row can touch, wherever they start.
int spans_of(int n) { return (n + kKvPage - 2) / kKvPage + 1; }

template <int D>
void append_d(const KvAppendArgs& a, unsigned kv_blocks, unsigned blocks, hipStream_t st) {
  const int spans = spans_of(a.batch.max_q);
  if (a.type == TERN_F32)
    tern_kv_append_kernel<D, TERN_F32><<<dim3(blocks), dim3(kThreads), 0, st>>>(a, spans, kv_blocks);
  else
    tern_kv_append_kernel<D, TERN_BF16><<<dim3(blocks), dim3(kThreads), 0, st>>>(a, spans, kv_blocks);
}

}  // namespace

// Workgroups of the append, for the host's check of the grid.
int64_t kv_append_blocks(const KvAppendArgs& a, int64_t* kv_blocks) {
  *kv_blocks = (int64_t)spans_of(a.batch.max_q) * a.cache.heads * 2 * a.batch.seqs;
  return *kv_blocks + (a.q ? ((int64_t)a.tokens * a.q_heads * (a.cache.dim / 8) + kThreads - 1) / kThreads : 0);
}
int64_t kv_read_blocks(const KvReadArgs& a) {
  return (int64_t)spans_of(a.batch.max_q) * a.cache.heads * 2 * a.batch.seqs;
}

int launch_kv_append(const KvAppendArgs& a, void* stream) {
  int64_t kv_blocks;
  const int64_t blocks = kv_append_blocks(a, &kv_blocks);
  hipStream_t st = (hipStream_t)stream;
  switch (a.cache.dim) {
    case 64: append_d<64>(a, (unsigned)kv_blocks, (unsigned)blocks, st); break;
    case 128: append_d<128>(a, (unsigned)kv_blocks, (unsigned)blocks, st); break;
    default: append_d<256>(a, (unsigned)kv_blocks, (unsigned)blocks, st); break;
  }
  return kernel_launched((int)hipGetLastError(), TERN_KERNEL_KV_APPEND);
}

int launch_kv_read(const KvReadArgs& a, void* stream) {
  const dim3 grid((unsigned)kv_read_blocks(a)), block(kThreads);
  hipStream_t st = (hipStream_t)stream;
  const int spans = spans_of(a.batch.max_q);
  switch (a.cache.dim) {
    case 64: tern_kv_read_kernel<64><<<grid, block, 0, st>>>(a, spans); break;
    case 128: tern_kv_read_kernel<128><<<grid, block, 0, st>>>(a, spans); break;
    default: tern_kv_read_kernel<256><<<grid, block, 0, st>>>(a, spans); break;
  }
  return kernel_launched((int)hipGetLastError(), TERN_KERNEL_KV_READ);
}

}  // namespace tern
