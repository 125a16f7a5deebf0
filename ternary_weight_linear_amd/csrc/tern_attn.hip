// tern_attn.hip -- gfx950 kernels of tern_kv_attn: attention over the 8-bit
// paged key/value cache.
//
// One page (64 tokens, one key scale, one value scale per kv head) is one
// step. With R query rows (a row is one token and one query head of the kv
// head's group) a wave computes
//   S^T [64 tokens x R] = K Q^T,   O^T [d x R] += V^T P^T
// on v_mfma_f32_16x16x32_f16. Both products are taken transposed so that a
// query row is a column of every tile: lane & 15 holds the row, and its
// maximum, sum and rescaling factor stay in the lane. The rows of S^T that a
// lane holds (tokens 16 i + 4 g + 0..3 for its lane group g) are then exactly
// a B operand of the second product if V^T is read with its tokens in that
// order, which is the order the cache stores them in: P never moves between
// lanes.
//
// Codes become fp16 exactly (|code| <= 127): with u = code + 128 in the low
// byte, the fp16 pattern 0x6400 | u is 1024 + u, and one packed subtraction
// of 1152 leaves the code. A query row is brought to [1, 2) by a power of two,
// which keeps its 8 significant bits and every element down to 2^-24 of the
// largest. Scores are fp32; the key scale, the softmax scale and the row's
// power of two multiply them in one factor per lane and page.
//
// The value scale w of a page goes into the exponent: with the running
// maximum M of s + log2(w) (s: scores in powers of two), p' = 2^(s + log2 w -
// M) <= 1 weighs the codes as they are, the sum of weights collects p' / w,
// and no page's product has to be scaled by itself. p' enters the product
// times 2^15 as fp16: 11 bits down to 2^-29, so rounding p' once is the only
// rounding below fp32 here.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tern_device.h"
#include "tern_internal.h"

namespace tern {
namespace {
using namespace dev;

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr float kNone = -__builtin_inff();
constexpr float kLeastScale = 0x1p-100f;  // value scales below count as this
constexpr float kPScale = 0x1p15f;        // of p' in fp16
// Largest factor from a product of codes (below 2^16) to its score in powers
// of two: scores past 2^22 have no fp32 fraction left to tell keys apart, and
// bounding them keeps the rounding of a maximum below half a power of two, so
// p' stays in fp16.
constexpr float kMostFactor = 64.f;

// fp16 of the four codes of a dword, exactly.
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;
  const f16x2 bias = {(_Float16)-1152.f, (_Float16)-1152.f};
  const f16x2 a = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, u, 0x04010400u)) + bias;
  const f16x2 b = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, u, 0x04030402u)) + bias;
  lo = __builtin_bit_cast(uint32_t, a);
  hi = __builtin_bit_cast(uint32_t, b);
}
__device__ __forceinline__ f16x8 codes8(uint32_t w0, uint32_t w1) {
  uint32_t a, b, c, d;
  codes_f16(w0, a, b);
  codes_f16(w1, c, d);
  return __builtin_bit_cast(f16x8, u32x4{a, b, c, d});
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, f16x2));
}

// Maximum and sum over the four lanes that share lane & 15: the two halves
// of the wave, then the two rows of 16 of each half, by register swaps.
__device__ __forceinline__ float group_max(float v) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float group_sum(float v) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// A sequence as the kernels see it; n = 0 if its arrays contradict the bounds.
struct Seq {
  int row0, n, kv;
};
__device__ __forceinline__ Seq sequence(const KvAttnArgs& a, int s) {
  const int q0 = a.batch.q_begin[s], q1 = a.batch.q_begin[s + 1];
  const int kv = a.batch.kv_len[s];
  Seq r{q0, q1 - q0, kv};
  if (q0 < 0 || q1 > a.tokens || q1 < q0 || r.n > a.batch.max_q) r.n = 0;
  if (kv < 0 || kv > a.batch.max_kv) r.kv = 0;
  return r;
}

// Pages that rows of the tokens [t0, t1] of a sequence visit: the first
// `sink` pages, then [first, end).
struct Pages {
  int sink, first, end, count;
  __device__ __forceinline__ int at(int i) const { return i < sink ? i : first + (i - sink); }
};
__device__ __forceinline__ Pages pages_of(const KvAttnArgs& a, const Seq& s, int t0, int t1) {
  const int lo = s.kv - s.n + t0, hi = s.kv - s.n + t1;  // positions; below zero before the first key
  Pages p;
  p.end = hi < 0 ? 0 : hi / kKvPage + 1;
  p.first = a.window ? max(0, lo - a.window + 1) / kKvPage : 0;
  p.sink = min((a.sinks + kKvPage - 1) / kKvPage, p.first);
  p.first = min(p.first, p.end);
  p.sink = min(p.sink, p.first);
  p.count = p.sink + p.end - p.first;
  return p;
}

// Grid: (row block, kv head) x splits x seqs; 4 waves, wave w takes pages
// w, w + 4, ... of the split's run.
template <int D, int NT>
__global__ void __launch_bounds__(256, D * NT <= 64 ? 4 : D == 128 && NT == 1 ? 3 : D * NT <= 256 ? 2 : 1) tern_kv_attn_kernel(KvAttnArgs a, KvAttnPlan plan, float* part) {
  constexpr int C = D / 64;   // 64-wide chunks of a head
  constexpr int HT = D / 16;  // 16-wide row tiles of O^T
  constexpr int R = 16 * NT;
  extern __shared__ float lds[];  // 2 x (R x D + 2 R): partial results of two waves
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int heads = a.cache.heads, group = a.q_heads / heads;
  const int head = blockIdx.x % heads, block = blockIdx.x / heads;
  const int split = blockIdx.y, sid = blockIdx.z;
  const Seq seq = sequence(a, sid);
  const int rows = seq.n * group;
  const int r0 = block * R;
  if (r0 >= rows) return;
  const int rlast = min(r0 + R, rows) - 1;
  const Pages pages = pages_of(a, seq, r0 / group, rlast / group);
  const int begin = split * plan.chunk, end = min(pages.count, begin + plan.chunk);
  if (begin >= end && split > 0) return;
  const int splits = (pages.count + plan.chunk - 1) / plan.chunk;  // of this row block

  // Page ids and scales of this wave's next 64 pages, one a lane; then keys
  // and values, asked for one buffer ahead of their use: a page's 16-byte
  // loads (N of keys, N of values a lane) go through two buffers of B in turn,
  // and each buffer is refilled as soon as it has been used. Streamed once:
  // non-temporal.
  constexpr int N = D / 16, B = N < 8 ? N : 8, H = N / B;
  u32x4 buf[2][B];
  const int32_t* table = a.batch.page_table + (int64_t)sid * a.batch.table_width;
  int id = -1, steps = 0;
  float ks = 0.f, vs = 0.f;
  auto ids = [&](int base) {
    const int mine = base + wave + 4 * lane;
    steps = (min(end, base + 256) - base - wave + 3) >> 2;
    id = mine < end ? table[pages.at(mine)] : -1;
  };
  auto scales = [&]() {
    if (id >= a.cache.pages) id = -1;
    ks = vs = 0.f;
    if (id >= 0) {
      const int64_t ph = (int64_t)id * heads + head;
      ks = a.cache.k_scale[ph];
      vs = a.cache.v_scale[ph];
    }
  };
  // Part h (0..2H-1: keys, then values) of step i's page into its buffer. A
  // page outside the cache reads page 0 instead, and is masked.
  auto ask = [&](int i, int h) {
    const int pid = max(__builtin_amdgcn_readlane(id, i), 0);
    const int64_t off = ((int64_t)pid * heads + head) * (kKvPage * D);
    if (h < H) {
      const int8_t* p = a.cache.k + off + n * D + 16 * g;
#pragma unroll
      for (int j = 0; j < B; ++j) {
        const int x = h * B + j;  // tokens 16 (x / C) .., elements 64 (x % C) ..
        buf[h & 1][j] = __builtin_nontemporal_load((const u32x4*)(p + 16 * (x / C) * D + 64 * (x % C)));
      }
    } else {
      const int8_t* p = a.cache.v + off + n * kKvPage + 16 * g;
#pragma unroll
      for (int j = 0; j < B; ++j)
        buf[h & 1][j] = __builtin_nontemporal_load((const u32x4*)(p + 16 * ((h - H) * B + j) * kKvPage));
    }
  };
  auto start = [&]() {
    scales();
    if (steps > 0) {
      ask(0, 0);
      ask(0, 1);
    }
  };
  // The chain of dependent loads at the start (lengths, page ids, scales and
  // codes) is what a short call waits for: everything is asked for as soon as
  // its address is known, the query rows between the ids and the codes.
  ids(begin);
  u32x4 raw[NT][C][2];
  int pos[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int rr = min(r0 + 16 * t + n, rows - 1);
    const int tok = rr / group, h = head * group + rr % group;
    pos[t] = seq.kv - seq.n + tok;
    const uint16_t* q = a.q + (int64_t)(seq.row0 + tok) * a.q_stride + (int64_t)h * D;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int k = 0; k < 2; ++k) raw[t][c][k] = *(const u32x4*)(q + 64 * c + 16 * g + 8 * k);
  }
  __builtin_amdgcn_sched_barrier(0);
  start();
  __builtin_amdgcn_sched_barrier(0);

  // The query rows as fp16 operands, each brought to [1, 2) by a power of two.
  f16x8 qf[NT][C][2];
  float qs[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    uint32_t m = 0;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          m = max(m, max((raw[t][c][k][i] << 16) & 0x7fff0000u, raw[t][c][k][i] & 0x7fff0000u));
    m = __float_as_uint(group_max(__uint_as_float(min(m, 0x7f800000u))));  // a NaN takes infinity's exponent
    // 2^e <= max|q| < 2^(e+1); rows of zeros and of subnormals take e = -126
    const int e = min(max((int)(m >> 23) - 127, -126), 126);
    const float down = __uint_as_float((uint32_t)(127 - e) << 23);
    qs[t] = a.scale * 1.4426950408889634f * __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          qf[t][c][k][2 * i] = (_Float16)(bf16_lo(raw[t][c][k][i]) * down);
          qf[t][c][k][2 * i + 1] = (_Float16)(bf16_hi(raw[t][c][k][i]) * down);
        }
  }
  const int pos_min = seq.kv - seq.n + r0 / group, pos_max = seq.kv - seq.n + rlast / group;

  f32x4 o[NT][HT];
  float M[NT], L[NT];  // L: this lane's share of the sum
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    M[t] = kNone;
    L[t] = 0.f;
#pragma unroll
    for (int i = 0; i < HT; ++i) o[t][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  for (int base = begin; base < end;) {
    vs = vs < kLeastScale ? kLeastScale : vs;
    const float lv = __builtin_amdgcn_logf(vs), iv = 1.0f / (vs * kPScale);
    for (int i = 0; i < steps; ++i) {
      // What follows part h in its buffer: part h + 2 of this page or the next one's.
      auto refill = [&](int h) {
        if (h + 2 < 2 * H)
          ask(i, h + 2);
        else if (i + 1 < steps)
          ask(i + 1, h + 2 - 2 * H);
      };
      const bool absent = __builtin_amdgcn_readlane(id, i) < 0;
      const float ksc = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(ks), i));
      const float lvs = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(lv), i));
      const float ivs = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(iv), i));
      const int j0 = pages.at(base + wave + 4 * i) * kKvPage;

      f32x4 s[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int b = 0; b < 4; ++b) s[t][b] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int h = 0; h < H; ++h) {
#pragma unroll
        for (int j = 0; j < B; ++j) {
          const int x = h * B + j, b = x / C, c = x % C;
          const u32x4 w = buf[h & 1][j];
          const f16x8 k0 = codes8(w[0], w[1]), k1 = codes8(w[2], w[3]);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            s[t][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k0, qf[t][c][0], s[t][b], 0, 0, 0);
            s[t][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k1, qf[t][c][1], s[t][b], 0, 0, 0);
          }
        }
        refill(h);
      }

      // Whether every row sees the whole page.
      const bool whole = !absent && j0 + kKvPage - 1 <= pos_min &&
                         (!a.window || j0 > pos_max - a.window || j0 + kKvPage <= a.sinks);
      f16x8 pf[NT][2];
      float alpha[NT];
      auto softmax = [&](auto masked) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float f = ksc * qs[t];
          f = f > kMostFactor ? kMostFactor : f;  // NaN stays
          float mx = kNone;
          bool see[4][4];
#pragma unroll
          for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if constexpr (decltype(masked)::value) {
                const int j = j0 + 16 * b + 4 * g + e;
                see[b][e] = !absent && j <= pos[t] && (!a.window || j > pos[t] - a.window || j < a.sinks);
                mx = fmaxf(mx, see[b][e] ? s[t][b][e] : kNone);
              } else {
                mx = fmaxf(mx, s[t][b][e]);
              }
            }
          mx = group_max(mx);
          const float top = mx == kNone ? kNone : __builtin_fmaf(mx, f, lvs);
          const float Mn = fmaxf(M[t], top);
          const float base2 = Mn == kNone ? 0.f : Mn;
          alpha[t] = __builtin_amdgcn_exp2f(M[t] - base2);
          M[t] = Mn;
          const float add = (lvs - base2) + 15.f;  // p' in fp16 stands times 2^15
          float sum = 0.f;
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            float p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              p[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][b][e], f, add));
              if constexpr (decltype(masked)::value) p[e] = see[b][e] ? p[e] : 0.f;
              sum += p[e];
            }
            const u32x2 w = {pack_f16(p[0], p[1]), pack_f16(p[2], p[3])};
            const f16x4 v = __builtin_bit_cast(f16x4, w);
#pragma unroll
            for (int e = 0; e < 4; ++e) pf[t][b >> 1][4 * (b & 1) + e] = v[e];
          }
          L[t] = __builtin_fmaf(L[t], alpha[t], sum * ivs);
        }
      };
      if (whole)
        softmax(std::false_type{});
      else
        softmax(std::true_type{});
#pragma unroll
      for (int t = 0; t < NT; ++t)
        if (__any(alpha[t] != 1.f)) {  // a maximum moved (or a row is NaN)
#pragma unroll
          for (int x = 0; x < HT; ++x) o[t][x] *= alpha[t];
        }
#pragma unroll
      for (int h = 0; h < H; ++h) {
#pragma unroll
        for (int j = 0; j < B; ++j) {
          const int x = h * B + j;
          const u32x4 w = buf[(H + h) & 1][j];
          const f16x8 v0 = codes8(w[0], w[1]), v1 = codes8(w[2], w[3]);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            o[t][x] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, pf[t][0], o[t][x], 0, 0, 0);
            o[t][x] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, pf[t][1], o[t][x], 0, 0, 0);
          }
        }
        refill(H + h);
      }
    }
    base += 256;
    if (base < end) {
      ids(base);
      start();
    }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) L[t] = group_sum(L[t]);

  // Join the four waves: 2 and 3 into 0 and 1, then 1 into 0.
  constexpr int kSlot = R * D + 2 * R;
#pragma unroll
  for (int from = 2; from >= 1; from >>= 1) {
    const int slot = wave % from;
    float* ml = lds + slot * kSlot + R * D;
    if (wave >= from && wave < 2 * from) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int h = 0; h < HT; ++h)
          *(f32x4*)(lds + slot * kSlot + ((t * HT + h) * 64 + lane) * 4) = o[t][h];
        if (g == 0) ml[16 * t + n] = M[t], ml[R + 16 * t + n] = L[t];
      }
    }
    __syncthreads();
    if (wave < from) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float m2 = ml[16 * t + n], l2 = ml[R + 16 * t + n];
        const float Mn = fmaxf(M[t], m2), b = Mn == kNone ? 0.f : Mn;
        const float x = __builtin_amdgcn_exp2f(M[t] - b), y = __builtin_amdgcn_exp2f(m2 - b);
        M[t] = Mn;
        L[t] = L[t] * x + l2 * y;
#pragma unroll
        for (int h = 0; h < HT; ++h)
          o[t][h] = o[t][h] * x + *(const f32x4*)(lds + slot * kSlot + ((t * HT + h) * 64 + lane) * 4) * y;
      }
    }
    __syncthreads();
  }
  if (wave != 0) return;
  // Row of the lane in [tokens][q_heads], or -1 past the sequence's last.
  auto row_at = [&](int t) -> int64_t {
    const int r = r0 + 16 * t + n;
    return r < rows ? (int64_t)(seq.row0 + r / group) * a.q_heads + head * group + r % group : -1;
  };
  if (splits <= 1) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int64_t at = row_at(t);
      if (at < 0) continue;
      const float inv = L[t] == 0.f ? 0.f : 1.0f / (L[t] * kPScale);
      uint16_t* out = a.out + at * D + 4 * g;
#pragma unroll
      for (int h = 0; h < HT; ++h)
        *(uint2*)(out + 16 * h) =
            uint2{pack_bf16(o[t][h][0] * inv, o[t][h][1] * inv), pack_bf16(o[t][h][2] * inv, o[t][h][3] * inv)};
    }
    return;
  }
  const int64_t all = (int64_t)a.tokens * a.q_heads;
  float* po = part + (int64_t)split * all * D;
  float* pm = part + (int64_t)plan.splits * all * D + (int64_t)split * all * 2;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int64_t at = row_at(t);
    if (at < 0) continue;
#pragma unroll
    for (int h = 0; h < HT; ++h) *(f32x4*)(po + at * D + 16 * h + 4 * g) = o[t][h];
    if (g == 0) *(float2*)(pm + at * 2) = float2{M[t], L[t]};
  }
}

// Joins the runs of each row; one workgroup of 256 threads a row. Every
// D/4 threads add the runs s, s + G, ... of four elements each, and the G
// partial sums are added in order, so a row's result does not depend on timing.
template <int D>
__global__ void __launch_bounds__(256) tern_kv_attn_join_kernel(KvAttnArgs a, KvAttnPlan plan, const float* part) {
  constexpr int G = 1024 / D;
  __shared__ float weight[kKvMaxSplits];
  __shared__ float red[8];
  __shared__ f32x4 sums[256];
  const int heads = a.cache.heads, group = a.q_heads / heads;
  const Seq seq = sequence(a, blockIdx.z);
  const int tok = blockIdx.x, h = blockIdx.y;
  if (tok >= seq.n) return;
  const int r0 = (tok * group + h % group) / plan.rows * plan.rows;
  const int rlast = min(r0 + plan.rows, seq.n * group) - 1;
  const Pages pages = pages_of(a, seq, r0 / group, rlast / group);
  const int splits = (pages.count + plan.chunk - 1) / plan.chunk;
  if (splits <= 1) return;  // written by its workgroup
  const int64_t all = (int64_t)a.tokens * a.q_heads;
  const int64_t at = (int64_t)(seq.row0 + tok) * a.q_heads + h;
  const float2* pm = (const float2*)(part + (int64_t)plan.splits * all * D) + at;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float M = kNone;
  float2 ml[kKvMaxSplits / 256];
#pragma unroll
  for (int u = 0; u < kKvMaxSplits / 256; ++u) {
    const int s = threadIdx.x + 256 * u;
    ml[u] = s < splits ? pm[s * all] : float2{kNone, 0.f};
    M = fmaxf(M, ml[u].x);
  }
  for (int x = 1; x < 64; x <<= 1) M = fmaxf(M, __shfl_xor(M, x));
  if (lane == 0) red[wave] = M;
  __syncthreads();
  M = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  const float b = M == kNone ? 0.f : M;
  float L = 0.f;
#pragma unroll
  for (int u = 0; u < kKvMaxSplits / 256; ++u) {
    const int s = threadIdx.x + 256 * u;
    const float w = __builtin_amdgcn_exp2f(ml[u].x - b);
    if (s < splits) {
      weight[s] = w;
      L = __builtin_fmaf(ml[u].y, w, L);
    }
  }
  L = wave_sum(L);
  if (lane == 0) red[4 + wave] = L;
  __syncthreads();
  L = (red[4] + red[5]) + (red[6] + red[7]);
  const int e = threadIdx.x % (D / 4), grp = threadIdx.x / (D / 4);
  const f32x4* po = (const f32x4*)(part + at * D) + e;
  f32x4 o = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int s = grp; s < splits; s += G) o += po[s * all * (D / 4)] * weight[s];
  sums[threadIdx.x] = o;
  __syncthreads();
  if (grp != 0) return;
#pragma unroll
  for (int x = 1; x < G; ++x) o += sums[e + x * (D / 4)];
  const float inv = L == 0.f ? 0.f : 1.0f / (L * kPScale);
  *(uint2*)(a.out + at * D + 4 * e) = uint2{pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv)};
}

template <int D, int NT>
hipError_t go(const KvAttnArgs& a, const KvAttnPlan& p, float* part, hipStream_t st) {
  constexpr int lds = 2 * (16 * NT * D + 2 * 16 * NT) * 4;
  if (lds > 65536) {
    const hipError_t e = hipFuncSetAttribute((const void*)tern_kv_attn_kernel<D, NT>,
                                             hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  tern_kv_attn_kernel<D, NT><<<dim3(p.row_blocks * a.cache.heads, p.splits, a.batch.seqs), dim3(256), lds, st>>>(a, p, part);
  return hipGetLastError();
}

template <int D>
int launch(const KvAttnArgs& a, const KvAttnPlan& p, float* part, hipStream_t st) {
  const hipError_t e = p.rows == 16 ? go<D, 1>(a, p, part, st) : go<D, 2>(a, p, part, st);
  if (kernel_launched((int)e, TERN_KERNEL_KV_ATTN)) return (int)e;
  if (p.splits == 1) return 0;
  tern_kv_attn_join_kernel<D><<<dim3(a.batch.max_q, a.q_heads, a.batch.seqs), dim3(256), 0, st>>>(a, p, part);
  return kernel_launched((int)hipGetLastError(), TERN_KERNEL_KV_ATTN_JOIN);
}

}  // namespace

int launch_kv_attn(const KvAttnArgs& a, const KvAttnPlan& p, void* ws, void* stream) {
  hipStream_t st = (hipStream_t)stream;
  switch (a.cache.dim) {
    case 64: return launch<64>(a, p, (float*)ws, st);
    case 128: return launch<128>(a, p, (float*)ws, st);
    default: return launch<256>(a, p, (float*)ws, st);
  }
}

}  // namespace tern
