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
// which keeps the 8 significant bits of every element down to 2^-14 of the
// largest, fewer below, and none from 2^-25 on: an error of at most 2^-25 of the
// largest times a code, as fp32 makes in the sum. Scores are fp32; the key scale,
// the softmax scale and the row's power of two multiply them in one factor per
// lane and page.
//
// The value scale w of a page goes into the exponent: with the running
// maximum M of s + log2(w) (s: scores in powers of two), p' = 2^(s + log2 w -
// M) <= 1 weighs the codes as they are, the sum of weights collects p' / w,
// and no page's product has to be scaled by itself. p' enters the product
// times 2^15 as fp16: 11 bits down to 2^-29, so rounding p' once is the only
// rounding below fp32 here.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "tern_decoder.h"
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
// With a factor f from a product of codes (at most 2^16) to its score in powers
// of two up to this, scores stay below 2^22 and the rounding of a maximum below
// half a power of two, so p' stays in fp16. Steeper rows subtract the page's
// maximum from the products first.
constexpr float kSteep = 64.f;
// Largest such factor: products times this are finite.
constexpr float kMostFactor = 0x1p111f;

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

// Workgroup barrier that waits for this wave's LDS operations only, not for
// the codes on their way from memory, as __syncthreads() would.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_s_waitcnt(0xC07F);  // vmcnt 63 (no wait), expcnt 7, lgkmcnt 0
  asm volatile("s_barrier" ::: "memory");
}

// x, but what is computed from it stays where it stands: addresses of results
// are not made ahead of the page loop, whose registers they would take.
__device__ __forceinline__ int here(int x) {
  asm volatile("" : "+v"(x));
  return x;
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

// A unit is one block of `plan.rows` query rows of a sequence, for one kv head.
// Unit u of a head: sequence u / row_blocks, block u % row_blocks.
struct Unit {
  Seq seq;
  int rows, r0, rlast;  // rows of the sequence, first and last of the unit (rlast < r0: none)
  Pages pages;
};
__device__ __forceinline__ Unit unit_of(const KvAttnArgs& a, const KvAttnPlan& plan, int u) {
  const int group = a.q_heads / a.cache.heads;
  Unit x;
  x.seq = sequence(a, u / plan.row_blocks);
  x.rows = x.seq.n * group;
  x.r0 = u % plan.row_blocks * plan.rows;
  x.rlast = min(x.r0 + plan.rows, x.rows) - 1;
  if (x.rlast >= x.r0)
    x.pages = pages_of(a, x.seq, x.r0 / group, x.rlast / group);
  else
    x.pages = Pages{0, 0, 0, 0};
  return x;
}

// Balanced runs (plan.runs > 0). The pages of all units of a head, one unit
// after the other, are cut into runs of equal length, one a workgroup, so that
// sequences of any lengths load the machine evenly; a run that ends inside a
// unit leaves a partial result there, which the join kernel adds up. Lengths
// are only known on the device, so every workgroup computes the prefix sums
// of the units' pages itself, and the first leaves them for the join kernel:
//   head of the workspace: run length, then pre[0 .. units];
//   then partial sums [heads][runs][2][rows][D] and (maximum, sum) pairs
//   [heads][runs][2][rows][2]; a run's slot 0 holds the unit that it enters
//   in the middle, slot 1 the one that it begins and does not finish.
struct Run {
  int length, begin, end, unit;  // pages [begin, end) of the head, starting in `unit`
};
__device__ __forceinline__ Run make_runs(const KvAttnArgs& a, const KvAttnPlan& plan, int w, int* pre, int* ws) {
  const int units = a.batch.seqs * plan.row_blocks;
  const int per = (units + 255) >> 8, u0 = threadIdx.x * per;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int sum = 0;
  for (int u = u0; u < min(u0 + per, units); ++u) {
    const int c = unit_of(a, plan, u).pages.count;
    pre[u + 1] = c;
    sum += c;
  }
  int scan = sum;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(scan, d);
    if (lane >= d) scan += v;
  }
  int* tail = pre + units + 1;  // the four waves' sums, then the unit found
  if (lane == 63) tail[wave] = scan;
  __syncthreads();
  int at = scan - sum;
  for (int i = 0; i < wave; ++i) at += tail[i];
  const int total = (tail[0] + tail[1]) + (tail[2] + tail[3]);
  Run r;
  r.length = max(plan.least, (total + plan.runs - 1) / plan.runs);
  r.length = __builtin_amdgcn_readfirstlane(r.length);
  r.begin = __builtin_amdgcn_readfirstlane((int)min((int64_t)w * r.length, (int64_t)total));
  r.end = __builtin_amdgcn_readfirstlane((int)min((int64_t)r.begin + r.length, (int64_t)total));
  if (threadIdx.x == 0) pre[0] = 0;
  for (int u = u0; u < min(u0 + per, units); ++u) {
    const int c = pre[u + 1];
    if (at <= r.begin && r.begin < at + c) tail[4] = u;
    at += c;
    pre[u + 1] = at;
  }
  __syncthreads();
  r.unit = __builtin_amdgcn_readfirstlane(tail[4]);
  if (blockIdx.x == 0) {
    for (int u = threadIdx.x; u <= units; u += blockDim.x) ws[1 + u] = pre[u];
    if (threadIdx.x == 0) ws[0] = r.length;
  }
  return r;
}
__device__ __forceinline__ int64_t ws_head(const KvAttnArgs& a, const KvAttnPlan& plan) {  // in floats
  return ((int64_t)a.batch.seqs * plan.row_blocks + 2 + 63) / 64 * 64;
}

// Query rows of a wave: NT tiles of 16, lane & 15 the row of each.
template <int D, int NT>
struct Queries {
  static constexpr int C = D / 64;  // 64-wide chunks of a head
  u32x4 raw[NT][C][2];
  f16x8 op[NT][C][2];  // operands: elements 64 c + 16 g + 8 k ..
  float factor[NT];    // from a product of operands and codes to a score in powers of two, but for the key scale
  int pos[NT];         // the row's position

  // Asks for the rows from `row` of a sequence on; rows past its last repeat that.
  __device__ __forceinline__ void ask(const KvAttnArgs& a, const Seq& seq, int row, int rows, int head, int group,
                                      int n, int g) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int rr = min(row + 16 * t + n, rows - 1);
      const int tok = rr / group, h = head * group + rr % group;
      pos[t] = seq.kv - seq.n + tok;
      const uint16_t* q = a.q + (int64_t)(seq.row0 + tok) * a.q_stride + (int64_t)h * D;
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int k = 0; k < 2; ++k) raw[t][c][k] = *(const u32x4*)(q + 64 * c + 16 * g + 8 * k);
    }
  }
  // fp16 operands, each row brought to [1, 2) by a power of two.
  __device__ __forceinline__ void make(float scale) {
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
      // A row with an infinite element has only infinite and NaN scores, so no
      // result: its operands become NaN, since a score of -inf would pass for hidden.
      const float down = __uint_as_float(m == 0x7f800000u ? 0x7fc00000u : (uint32_t)(127 - e) << 23);
      // finite, so that a page of zero keys has scores of zero
      factor[t] = fminf(scale * 1.4426950408889634f * __uint_as_float((uint32_t)(127 + e) << 23), 0x1p127f);
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            op[t][c][k][2 * i] = (_Float16)(bf16_lo(raw[t][c][k][i]) * down);
            op[t][c][k][2 * i + 1] = (_Float16)(bf16_hi(raw[t][c][k][i]) * down);
          }
    }
  }
  // Whether some row's factor with key scale k is above kSteep.
  __device__ __forceinline__ bool steep(float k) const {
    bool any = false;
#pragma unroll
    for (int t = 0; t < NT; ++t) any |= k * factor[t] > kSteep;
    return __any(any);
  }
};

// What a page multiplies with: key scale, log2 of the value scale w and
// 2^-15 / w; a page outside the cache is absent.
struct PageScales {
  float k, log_v, inv_v;
  bool absent;
};

// 2^-15 / w. A NaN scale makes the rows NaN that see the page through its
// logarithm; here it counts as 0, for the rows that do not (0 * NaN).
__device__ __forceinline__ float weight_of(float w) { return w == w ? 1.0f / w * (1.0f / kPScale) : 0.f; }

// Softmax of a page's scores s for the 16 rows of one tile: running maximum M
// and sum L, the factor alpha for what was summed before, and the second
// product's operands p. MASKED: some row does not see the whole page.
// STEEP: some row's factor may be above kSteep.
template <bool MASKED, bool STEEP>
__device__ __forceinline__ void page_softmax(f32x4 (&s)[4], const PageScales& w, float factor, int pos, int j0, int g,
                                             int window, int sinks, float& M, float& L, float& alpha, f16x8 (&p)[2]) {
  float f = w.k * factor;
  f = f > kMostFactor ? kMostFactor : f;  // NaN stays
  float mx = kNone;
  // Masked: element 16 b + e of this lane's tokens is seen up to `last`, but
  // for those from `hide` on and before `show` (past the sinks, before the window).
  const int at = j0 + 4 * g;
  const int last = w.absent ? -1 : pos - at, show = window ? pos - window + 1 - at : 0, hide = window ? sinks - at : 64;
#pragma unroll
  for (int b = 0; b < 4; ++b)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (MASKED) {
        const int x = 16 * b + e;
        s[b][e] = x > last || (x >= hide && x < show) ? kNone : s[b][e];
      }
      mx = fmaxf(mx, s[b][e]);
    }
  mx = group_max(mx);
  const float top = mx == kNone ? kNone : __builtin_fmaf(mx, f, w.log_v);
  const float Mn = fmaxf(M, top);
  const float base = Mn == kNone ? 0.f : Mn;
  // Of pages whose value scales lie far apart the smaller one's p' vanish beside
  // the other's, but p' / w does not. So the sum of weights takes alpha in two
  // steps, and a page far below the maximum raises its p' to at most 2^-100 and
  // its sum back: neither leaves fp32 on the way.
  const float root = __builtin_amdgcn_exp2f(0.5f * (M - base));
  alpha = root * root;
  M = Mn;
  float add = (w.log_v - base) + 15.f;  // p' in fp16 stands times 2^15
  if constexpr (STEEP) {
    // (s - mx) f + (top - base) has two terms that are never positive, whatever
    // f is. Rows with a smaller factor keep their form, so that no row's result
    // depends on its neighbours.
    const bool steep = f > kSteep;
    const float r = steep && mx != kNone ? mx : 0.f;
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[b][e] -= r;
    add = steep ? (top - base) + 15.f : add;
  }
  const float lift = __builtin_amdgcn_fmed3f((base - top) - 100.f, 0.f, 124.f);
  add += lift;
  float sum = 0.f;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    float x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[b][e], f, add));
      if constexpr (MASKED) x[e] = s[b][e] == kNone ? 0.f : x[e];  // also where f is NaN
      sum += x[e];
    }
    const u32x2 h = {pack_f16(x[0], x[1]), pack_f16(x[2], x[3])};
    const f16x4 v = __builtin_bit_cast(f16x4, h);
#pragma unroll
    for (int e = 0; e < 4; ++e) p[b >> 1][4 * (b & 1) + e] = v[e];
  }
  L = __builtin_fmaf(L * root, root, sum * w.inv_v * __builtin_amdgcn_exp2f(-lift));
}

__device__ __forceinline__ float lane_float(float v, int lane) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), lane));
}

// A row's result, or its partial sums, from the lanes that hold it (four
// consecutive elements of every 16).
template <int D>
__device__ __forceinline__ void write_row(const KvAttnArgs& a, const f32x4 (&o)[D / 16], float L, int64_t at, int g) {
  const float inv = L == 0.f ? 0.f : 1.0f / L * (1.0f / kPScale);  // L kPScale may pass fp32
  uint16_t* out = a.out + at * D + 4 * g;
#pragma unroll
  for (int h = 0; h < D / 16; ++h)
    *(uint2*)(out + 16 * h) = uint2{pack_bf16(o[h][0] * inv, o[h][1] * inv), pack_bf16(o[h][2] * inv, o[h][3] * inv)};
}
template <int D>
__device__ __forceinline__ void write_part(float* po, float* pm, const f32x4 (&o)[D / 16], float M, float L, int row,
                                           int g) {
#pragma unroll
  for (int h = 0; h < D / 16; ++h) *(f32x4*)(po + row * D + 16 * h + 4 * g) = o[h];
  if (g == 0) *(float2*)(pm + row * 2) = float2{M, L};
}

// Few query rows. Grid: kv heads x units, or kv heads x runs. 4 waves; wave w
// takes pages w, w + 4, ... of what the workgroup visits of a unit.
//
// Bound by HBM: every code is read once, straight to the registers of the wave
// that uses it. About 460 vector instructions a page (conversion 320, softmax
// 140) run beside the 16 KB of a page at d = 128. One workgroup a compute unit
// with two pages' halves in flight a wave is enough (8 waves a workgroup, or
// more workgroups, were no faster). One sequence of 131072 tokens: 46 us =
// 5.8 TB/s (a read of as many bytes without other work: 39 us); 32 sequences
// of 1024 to 8192 tokens: 56 us = 5.5 TB/s; both + 5 us for the join. 16
// sequences x 4 tokens: 27 us for 80 MB, of which about 10 are the start
// (lengths, prefix sums, page ids, first codes) and end of a workgroup.
template <int D, int NT>
__global__ void __launch_bounds__(256, D * NT <= 64 ? 4 : D * NT <= 256 ? 2 : 1)
    tern_kv_attn_kernel(KvAttnArgs a, KvAttnPlan plan, float* ws) {
  constexpr int C = D / 64;   // 64-wide chunks of a head
  constexpr int HT = D / 16;  // 16-wide row tiles of O^T
  constexpr int R = 16 * NT;
  constexpr int kSlot = R * D + 2 * R;  // a wave's partial result
  extern __shared__ float lds[];        // two of those; with runs, the prefix sums follow
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int heads = a.cache.heads, group = a.q_heads / heads;
  const int head = blockIdx.x % heads, w = blockIdx.x / heads;
  const int* pre = (const int*)(lds + 2 * kSlot);
  Run run{0, 0, 0, w};
  if (plan.runs) {
    run = make_runs(a, plan, w, (int*)(lds + 2 * kSlot), (int*)ws);
    if (run.begin >= run.end) return;
  }
  for (int u = run.unit, from = run.begin;;) {
    const Unit unit = unit_of(a, plan, u);
    if (unit.rlast < unit.r0) return;  // only without runs: no pages, no run here
    const Seq seq = unit.seq;
    const Pages pages = unit.pages;
    const int r0 = unit.r0, rows = unit.rows, rlast = unit.rlast;
    const int begin = plan.runs ? __builtin_amdgcn_readfirstlane(from - pre[u]) : 0;
    const int end = plan.runs ? min(pages.count, begin + run.end - from) : pages.count;

    // Page ids and scales of this wave's next 64 pages, one a lane; then keys
    // and values, asked for one buffer ahead of their use: a page's 16-byte
    // loads (N of keys, N of values a lane) go through two buffers of B in turn,
    // and each buffer is refilled as soon as it has been used. Streamed once:
    // non-temporal.
    constexpr int N = D / 16, B = N < 8 ? N : 8, H = N / B;
    u32x4 buf[2][B];
    const int32_t* table = a.batch.page_table + (int64_t)(u / plan.row_blocks) * a.batch.table_width;
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
    // page outside the cache, and one past the last step, are buffers of no
    // bytes: they read as zeros and cost no traffic, and every step issues the
    // same loads, so that a wait for one of them never waits for a later one.
    auto ask = [&](int i, int h) {
      const int pid = i < steps ? __builtin_amdgcn_readlane(id, i) : -1;
      const int64_t off = ((int64_t)pid * heads + head) * (kKvPage * D);
      const rsrc_t page = make_rsrc((h < H ? a.cache.k : a.cache.v) + off, pid < 0 ? 0 : kKvPage * D);
      const int lane_at = h < H ? n * D + 16 * g : n * kKvPage + 16 * g;
#pragma unroll
      for (int j = 0; j < B; ++j) {
        const int x = h % H * B + j;  // keys: tokens 16 (x / C) .., elements 64 (x % C) ..; values: elements 16 x ..
        const int at = h < H ? 16 * (x / C) * D + 64 * (x % C) : 16 * x * kKvPage;
        buf[h & 1][j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(page, lane_at, at, kAuxNontemporal));
      }
    };
    auto start = [&]() {
      scales();
      ask(0, 0);
      ask(0, 1);
    };
    // The chain of dependent loads at the start (lengths, page ids, scales and
    // codes) is what a short call waits for: everything is asked for as soon as
    // its address is known, the query rows between the ids and the codes.
    ids(begin);
    Queries<D, NT> q;
    q.ask(a, seq, r0, rows, head, group, n, g);
    __builtin_amdgcn_sched_barrier(0);
    start();
    __builtin_amdgcn_sched_barrier(0);
    q.make(a.scale);
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
      ks += ks - ks;  // an infinite scale becomes NaN, which the bound of the factor lets through
      vs = vs < kLeastScale ? kLeastScale : vs;
      const float lv = __builtin_amdgcn_logf(vs), iv = weight_of(vs);
      for (int i = 0; i < steps; ++i) {
        // What follows part h in its buffer: part h + 2 of this page or the next one's.
        auto refill = [&](int h) {
          if (h + 2 < 2 * H)
            ask(i, h + 2);
          else
            ask(i + 1, h + 2 - 2 * H);
        };
        const PageScales w{lane_float(ks, i), lane_float(lv, i), lane_float(iv, i), __builtin_amdgcn_readlane(id, i) < 0};
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
            const u32x4 x16 = buf[h & 1][j];
            const f16x8 k0 = codes8(x16[0], x16[1]), k1 = codes8(x16[2], x16[3]);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              s[t][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k0, q.op[t][c][0], s[t][b], 0, 0, 0);
              s[t][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k1, q.op[t][c][1], s[t][b], 0, 0, 0);
            }
          }
          refill(h);
        }

        // Whether every row sees the whole page.
        const bool whole = !w.absent && j0 + kKvPage - 1 <= pos_min &&
                           (!a.window || j0 > pos_max - a.window || j0 + kKvPage <= a.sinks);
        f16x8 pf[NT][2];
        float alpha[NT];
        // The form for steep rows always: its 16 subtractions a tile hide behind the
        // loads, a branch to it costs registers (16 x 4 tokens: 30.0 us against
        // 31.5; the other cases within 0.5 %).
        auto softmax = [&](auto masked) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
            page_softmax<decltype(masked)::value, true>(s[t], w, q.factor[t], q.pos[t], j0, g, a.window, a.sinks, M[t], L[t],
                                                        alpha[t], pf[t]);
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
            const u32x4 x16 = buf[(H + h) & 1][j];
            const f16x8 v0 = codes8(x16[0], x16[1]), v1 = codes8(x16[2], x16[3]);
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
    const int at = here(lane), n1 = at & 15, g1 = at >> 4;
#pragma unroll
    for (int half = 2; half >= 1; half >>= 1) {
      float* slot = lds + wave % half * kSlot;
      float* ml = slot + R * D;
      if (wave >= half && wave < 2 * half) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
          for (int h = 0; h < HT; ++h) *(f32x4*)(slot + ((t * HT + h) * 64 + at) * 4) = o[t][h];
          if (g1 == 0) ml[16 * t + n1] = M[t], ml[R + 16 * t + n1] = L[t];
        }
      }
      __syncthreads();
      if (wave < half) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const float m2 = ml[16 * t + n1], l2 = ml[R + 16 * t + n1];
          const float Mn = fmaxf(M[t], m2), b = Mn == kNone ? 0.f : Mn;
          const float x = __builtin_amdgcn_exp2f(M[t] - b), y = __builtin_amdgcn_exp2f(m2 - b);
          const float M0 = M[t];
          M[t] = Mn;
          const float rx = __builtin_amdgcn_exp2f(0.5f * (M0 - b)), ry = __builtin_amdgcn_exp2f(0.5f * (m2 - b));
          L[t] = L[t] * rx * rx + l2 * ry * ry;
#pragma unroll
          for (int h = 0; h < HT; ++h)
            o[t][h] = o[t][h] * x + *(const f32x4*)(slot + ((t * HT + h) * 64 + at) * 4) * y;
        }
      }
      __syncthreads();
    }
    if (wave == 0) {
      const bool whole = begin == 0 && end == pages.count;
      const int64_t slot = ((int64_t)head * plan.runs + w) * 2 + (begin == 0);
      float* po = ws + ws_head(a, plan) + slot * R * D;
      float* pm = ws + ws_head(a, plan) + (int64_t)heads * plan.runs * 2 * R * D + slot * R * 2;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int r = r0 + 16 * t + n1;
        if (r >= rows) continue;
        if (whole)
          write_row<D>(a, o[t], L[t], (int64_t)(seq.row0 + r / group) * a.q_heads + head * group + r % group, g1);
        else
          write_part<D>(po, pm, o[t], M[t], L[t], 16 * t + n1, g1);
      }
    }
    if (!plan.runs) return;
    from += end - begin;
    if (from >= run.end) return;
    do ++u;
    while (pre[u + 1] == pre[u]);  // the next unit with pages: there is one before run.end
    u = __builtin_amdgcn_readfirstlane(u);
  }
}

// Many query rows: a unit of 128 rows, 32 a wave, whose waves share each
// page's codes. Bound by instruction issue: a page costs a wave 64 matrix
// products (1024 cycles), about 340 vector instructions (1480) and 32 LDS
// reads, and they overlap little: leaving out any one of conversion, exp,
// either product or the LDS reads of a copy gains 6 to 16 % each, and a
// software pipeline that lays one page's softmax between the next page's
// products gained 4 % at d = 128 and lost 5 % at 256. 1024 tokens x 40 heads of
// 128 on 8192 keys: 209 us with the join (769 TFLOP/s; a library fp16 product
// of 8192^3 runs at 1165), of which the join takes 14. The workgroup turns the codes into fp16 operands once, in LDS
// (one page ahead: two buffers, one barrier a page), so that the conversion
// costs a quarter of what it costs a wave by itself; the operands lie in the
// order in which the lanes read them (64 lanes x 16 bytes each), free of bank
// conflicts both ways.
template <int D>
__global__ void __launch_bounds__(256, D == 256 ? 1 : 2) tern_kv_attn_tile_kernel(KvAttnArgs a, KvAttnPlan plan, float* ws) {
  constexpr int NT = 2, R = 128;
  constexpr int C = D / 64, HT = D / 16;
  constexpr int N = D / 16;           // 16-byte loads of a page's keys, or values, by one wave
  constexpr int kPage = 2 * N * 128;  // u32x4 of a buffer: keys, then values, two operands a load
  extern __shared__ u32x4 tiles[];    // two buffers; with runs, the prefix sums follow
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int heads = a.cache.heads, group = a.q_heads / heads;
  const int head = blockIdx.x % heads, w = blockIdx.x / heads;
  int* const pre = (int*)(tiles + 2 * kPage);
  Run run{0, 0, 0, a.batch.seqs * plan.row_blocks - 1 - w};  // without runs: the last rows, which see most, first
  if (plan.runs) {
    run = make_runs(a, plan, w, pre, (int*)ws);
    if (run.begin >= run.end) return;
  }
  for (int u = run.unit, from = run.begin;;) {
    const Unit unit = unit_of(a, plan, u);
    if (unit.rlast < unit.r0) return;  // only without runs: no pages, no run here
    const Seq seq = unit.seq;
    const Pages pages = unit.pages;
    const int rows = unit.rows, r0 = unit.r0 + 32 * wave;  // the wave's own rows from here on
    const int begin = plan.runs ? __builtin_amdgcn_readfirstlane(from - pre[u]) : 0;
    const int end = plan.runs ? min(pages.count, begin + run.end - from) : pages.count;

    Queries<D, NT> q;
    q.ask(a, seq, r0, rows, head, group, n, g);
    const int32_t* table = a.batch.page_table + (int64_t)(u / plan.row_blocks) * a.batch.table_width;
    // Ids and scales of 64 pages, one a lane; 62 steps are taken with them,
    // since codes are asked for two pages ahead.
    int id = -1;
    float ks = 0.f, lv = 0.f, iv = 0.f;
    auto ids = [&](int base) {
      const int mine = base + lane;
      id = mine < end ? table[pages.at(mine)] : -1;
      if (id >= a.cache.pages) id = -1;
      float vs = 0.f;
      ks = 0.f;
      if (id >= 0) {
        const int64_t ph = (int64_t)id * heads + head;
        ks = a.cache.k_scale[ph];
        ks += ks - ks;  // an infinite scale becomes NaN, which the bound of the factor lets through
        vs = a.cache.v_scale[ph];
      }
      vs = vs < kLeastScale ? kLeastScale : vs;
      lv = __builtin_amdgcn_logf(vs);
      iv = weight_of(vs);
    };
    // The wave's quarter of a page's codes: loads wave, wave + 4, ... of keys
    // and of values. A page that is absent, or past the end, reads as zeros.
    u32x4 raw[2][N / 4];
    auto ask = [&](int i) {
      const int pid = __builtin_amdgcn_readlane(id, i);
      const int64_t off = ((int64_t)pid * heads + head) * (kKvPage * D);
      const rsrc_t kr = make_rsrc(a.cache.k + off, pid < 0 ? 0 : kKvPage * D);
      const rsrc_t vr = make_rsrc(a.cache.v + off, pid < 0 ? 0 : kKvPage * D);
#pragma unroll
      for (int j = 0; j < N / 4; ++j) {
        const int x = wave + 4 * j;
        raw[0][j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                  kr, n * D + 16 * g, 16 * (x / C) * D + 64 * (x % C), 0));
        raw[1][j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                  vr, n * kKvPage + 16 * g, 16 * x * kKvPage, 0));
      }
    };
    auto convert = [&](u32x4* to) {
#pragma unroll
      for (int kv = 0; kv < 2; ++kv)
#pragma unroll
        for (int j = 0; j < N / 4; ++j) {
          const u32x4 c = raw[kv][j];
          u32x4* o = to + (kv * N + wave + 4 * j) * 128 + lane;
          o[0] = __builtin_bit_cast(u32x4, codes8(c[0], c[1]));
          o[64] = __builtin_bit_cast(u32x4, codes8(c[2], c[3]));
        }
    };
    ids(begin);
    ask(0);
    q.make(a.scale);
    const int wlast = min(r0 + 31, rows - 1);
    const int pos_min = seq.kv - seq.n + min(r0, rows - 1) / group, pos_max = seq.kv - seq.n + wlast / group;

    f32x4 o[NT][HT];
    float M[NT], L[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      M[t] = kNone;
      L[t] = 0.f;
#pragma unroll
      for (int i = 0; i < HT; ++i) o[t][i] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    convert(tiles);
    ask(1);
    int buffer = 0, base = begin;
    for (int i = begin; i < end; ++i) {
      if (i - base == 62) {
        base = i;
        ids(base);  // codes of page i + 1 are already on their way
      }
      const int at = i - base;
      lds_barrier();  // this page's operands are written, and the other buffer is read
      convert(tiles + (buffer ^ 1) * kPage);
      ask(at + 2);
      const u32x4* page = tiles + buffer * kPage + lane;
      buffer ^= 1;
      const PageScales ps{lane_float(ks, at), lane_float(lv, at), lane_float(iv, at), __builtin_amdgcn_readlane(id, at) < 0};
      const int j0 = pages.at(i) * kKvPage;
      // Pages that none of the wave's rows sees: after its last position, or
      // past the sinks and before its first window.
      if (r0 >= rows || ps.absent || j0 > pos_max ||
          (a.window && j0 + kKvPage - 1 <= pos_min - a.window && j0 >= a.sinks))
        continue;

      f32x4 s[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int b = 0; b < 4; ++b) s[t][b] = f32x4{0.f, 0.f, 0.f, 0.f};
      // Operands are read A loads ahead of their products, the first values'
      // before the softmax.
      constexpr int A = 4;
      f16x8 f[A][2];
      auto read = [&](int x) {
        f[x % A][0] = __builtin_bit_cast(f16x8, page[x * 128]);
        f[x % A][1] = __builtin_bit_cast(f16x8, page[x * 128 + 64]);
      };
#pragma unroll
      for (int x = 0; x < A; ++x) read(x);
#pragma unroll
      for (int x = 0; x < N; ++x) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          s[t][x / C] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f[x % A][0], q.op[t][x % C][0], s[t][x / C], 0, 0, 0);
          s[t][x / C] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f[x % A][1], q.op[t][x % C][1], s[t][x / C], 0, 0, 0);
        }
        read(x + A);
      }
      const bool whole = j0 + kKvPage - 1 <= pos_min &&
                         (!a.window || j0 > pos_max - a.window || j0 + kKvPage <= a.sinks);
      f16x8 pf[NT][2];
      float alpha[NT];
      auto softmax = [&](auto masked, auto steep) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
          page_softmax<decltype(masked)::value, decltype(steep)::value>(s[t], ps, q.factor[t], q.pos[t], j0, g, a.window,
                                                                        a.sinks, M[t], L[t], alpha[t], pf[t]);
      };
      // Bound by issue, so a branch: 1024 tokens on 8192 keys 211 us against 218 with
      // the form for steep rows always, 3 x 508 tokens with a window 109 against 112.
      if (q.steep(ps.k))
        softmax(std::true_type{}, std::true_type{});
      else if (whole)
        softmax(std::false_type{}, std::false_type{});
      else
        softmax(std::true_type{}, std::false_type{});
#pragma unroll
      for (int t = 0; t < NT; ++t)
        if (__any(alpha[t] != 1.f)) {  // a maximum moved (or a row is NaN)
#pragma unroll
          for (int x = 0; x < HT; ++x) o[t][x] *= alpha[t];
        }
#pragma unroll
      for (int x = 0; x < HT; ++x) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          o[t][x] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f[x % A][0], pf[t][0], o[t][x], 0, 0, 0);
          o[t][x] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f[x % A][1], pf[t][1], o[t][x], 0, 0, 0);
        }
        if (x + A < N) read(N + x + A);
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) L[t] = group_sum(L[t]);

    const int at = here(lane), n1 = at & 15, g1 = at >> 4;
    const bool whole = begin == 0 && end == pages.count;
    const int64_t slot = ((int64_t)head * plan.runs + w) * 2 + (begin == 0);
    float* po = ws + ws_head(a, plan) + slot * R * D;
    float* pm = ws + ws_head(a, plan) + (int64_t)heads * plan.runs * 2 * R * D + slot * R * 2;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int r = r0 + 16 * t + n1;
      if (r >= rows) continue;
      if (whole)
        write_row<D>(a, o[t], L[t], (int64_t)(seq.row0 + r / group) * a.q_heads + head * group + r % group, g1);
      else
        write_part<D>(po, pm, o[t], M[t], L[t], 32 * wave + 16 * t + n1, g1);
    }
    if (!plan.runs) return;
    from += end - begin;
    if (from >= run.end) return;
    do ++u;
    while (pre[u + 1] == pre[u]);  // the next unit with pages: there is one before run.end
    u = __builtin_amdgcn_readfirstlane(u);
    __syncthreads();  // the last page's operands are read
  }
}

// Joins the runs of a unit: D / 4 lanes a row, four elements each, that add
// the row's pieces in order, four pieces' loads at a time.
template <int D>
__global__ void __launch_bounds__(256) tern_kv_attn_join_kernel(KvAttnArgs a, KvAttnPlan plan, const float* ws, int count) {
  constexpr int W = D / 4;
  const int heads = a.cache.heads, group = a.q_heads / heads;
  const int l = threadIdx.x % W;
  const int i = blockIdx.x * (256 / W) + threadIdx.x / W;  // (row, head) of the unit
  if (i >= count) return;
  const int head = i % heads, row = i / heads, u = blockIdx.y;
  const int* pre = (const int*)ws + 1;
  const int length = pre[-1], p0 = pre[u], p1 = pre[u + 1];
  const Seq seq = sequence(a, u / plan.row_blocks);
  const int r = u % plan.row_blocks * plan.rows + row;
  if (r >= seq.n * group) return;
  const int first = p0 / length, last = p1 > p0 ? (p1 - 1) / length : first - 1;
  if (first == last) return;  // one piece: its workgroup wrote the result
  const int pieces = last - first + 1;  // 0: the row sees nothing
  const int64_t at = (int64_t)(seq.row0 + r / group) * a.q_heads + head * group + r % group;
  // Piece p is in slot 0 of run first + p, but for the first one, in slot 1.
  const int64_t slots = ((int64_t)head * plan.runs + first) * 2;
  const float* po = ws + ws_head(a, plan) + (slots * plan.rows + row) * D + 4 * l;
  const float* pm = ws + ws_head(a, plan) + (int64_t)heads * plan.runs * 2 * plan.rows * D + (slots * plan.rows + row) * 2;
  float M = kNone;
  for (int p = l; p < pieces; p += W) M = fmaxf(M, pm[(int64_t)(p ? 2 * p : 1) * plan.rows * 2]);
#pragma unroll
  for (int x = 1; x < W; x <<= 1) M = fmaxf(M, __shfl_xor(M, x));
  const float b = M == kNone ? 0.f : M;
  float L = 0.f;
  f32x4 o = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int q = 0; q < pieces; q += 4) {
    float2 ml[4];
    f32x4 f[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {  // past the last piece, that one again with no weight
      const int p = min(q + j, pieces - 1);
      const int64_t slot = (int64_t)(p ? 2 * p : 1) * plan.rows;
      ml[j] = *(const float2*)(pm + slot * 2);
      f[j] = *(const f32x4*)(po + slot * D);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float y = q + j < pieces ? __builtin_amdgcn_exp2f(ml[j].x - b) : 0.f;
      const float ry = q + j < pieces ? __builtin_amdgcn_exp2f(0.5f * (ml[j].x - b)) : 0.f;
      L = __builtin_fmaf(ml[j].y * ry, ry, L);
      o += f[j] * y;
    }
  }
  const float inv = L == 0.f ? 0.f : 1.0f / L * (1.0f / kPScale);  // L kPScale may pass fp32
  *(uint2*)(a.out + at * D + 4 * l) = uint2{pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv)};
}

template <class K>
hipError_t go(K* kernel, int lds, const KvAttnArgs& a, const KvAttnPlan& p, float* ws, hipStream_t st) {
  const int units = a.batch.seqs * p.row_blocks;
  if (p.runs) lds += (units + 6) * 4;
  if (lds > 65536) {
    const hipError_t e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  kernel<<<dim3(a.cache.heads * (p.runs ? p.runs : units)), dim3(256), lds, st>>>(a, p, ws);
  return hipGetLastError();
}

template <int D>
int launch(const KvAttnArgs& a, const KvAttnPlan& p, float* ws, hipStream_t st) {
  auto few = [](int rows) { return 2 * (rows * D + 2 * rows) * 4; };
  const hipError_t e = p.rows == 16   ? go(tern_kv_attn_kernel<D, 1>, few(16), a, p, ws, st)
                       : p.rows == 32 ? go(tern_kv_attn_kernel<D, 2>, few(32), a, p, ws, st)
                                      : go(tern_kv_attn_tile_kernel<D>, 2 * (D / 16) * 2 * 128 * 16, a, p, ws, st);
  if (kernel_launched((int)e, p.rows <= 32 ? TERN_KERNEL_KV_ATTN : TERN_KERNEL_KV_ATTN_TILE)) return (int)e;
  if (!p.runs) return 0;
  const int count = std::min(p.rows, a.q_heads / a.cache.heads * a.batch.max_q) * a.cache.heads, each = 1024 / D;
  const dim3 grid((count + each - 1) / each, a.batch.seqs * p.row_blocks);
  tern_kv_attn_join_kernel<D><<<grid, dim3(256), 0, st>>>(a, p, ws, count);
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
