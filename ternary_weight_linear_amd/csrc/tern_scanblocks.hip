// tern_scanblocks.hip -- gfx950 kernels of tern_scan for prompts: blocks of 32
// tokens through the matrix cores.
//
// With L[s] = sum_{i <= s} D[i] a from a block's start, and S the state there,
//   y[s] = exp(L[s]) C[s] S + sum_{t <= s} M[s][t] x[t] + d x[s],
//          M[s][t] = (C[s] . B[t]) exp(L[s] - L[t]) D[t],
//   S   <- exp(L[31]) S + sum_t B[t]^T (exp(L[31] - L[t]) D[t] x[t]).
//
// What does not depend on a state is made first, for all blocks at once: M of
// every head, and the factors exp(L) and exp(L[31] - L) D of every token. Then a
// workgroup takes 64 columns of x, of one or two heads of a group, in strips of
// 16 with two waves each, and goes along the blocks of a sequence's segment with S in
// registers, [state_dim / 2 x 16] a wave: the waves of a strip add up their parts of C S
// through LDS and make 16 rows of y each. All products are computed transposed, so that
// what one leaves is what the next takes, in the same lanes:
// v_mfma_f32_16x16x32_bf16 leaves row 4 (lane / 16) + r of column lane % 16 in
// register r, and two such results are an operand whose k runs in that order. S^T
// enters y^T = S^T C^T from its own registers, M^T lies in memory in the order of an
// operand's lanes, C in LDS in the order of k. B and x are read transposed from LDS.
//
// Sums, states and the factors exp() are fp32. B, C and x are bf16 as given. M and
// S enter y's products as two bf16 numbers each, which hold them to 2^-15, and the
// weighted x enters the next state, whose errors add up over a sequence, as three, which
// hold all of its 24 bits. (With one number each for M and S y is off by 2^-8 of its terms,
// as much as its own rounding where they do not cancel, and more where they do; 2048 tokens
// of 160 heads took 83 us.)
//
// Few workgroups (one sequence, few heads): the tokens of a sequence are cut
// into segments. A launch computes each segment's own state from zeros and its
// decay, the next puts the states at the segments' starts together in order.
//
// Bound by the issue of each workgroup's chain through a block (about 1.27 us for 64
// columns x 128 rows: loads to LDS, products, rounding, a barrier), which
// few workgroups cannot hide; the matrix cores and HBM are far from full. Measured:
// 2048 tokens of 160 heads of 64 x 128 in 15 + 82 us (13 us of matrix products at the whole
// chip's rate, 21 us of traffic); 3 x 509 of 40 heads of 128 x 64 in 5 + 20; 8192 of 20
// heads of 64 x 128 in 12 segments, 9 + 19 + 6 + 33. Products of 32 x 32 x 16 with 128
// columns a workgroup (with one number each for M and S) took 65 us against 82 for 512 tokens of
// 1024 heads, and were slower where units are few.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tern_recurrent.h"

namespace tern {
namespace {
using namespace dev;

typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int kBlock = kScanBlock;
constexpr float kLog2e = 1.44269504f;

__device__ __forceinline__ f32x4 mfma(const u32x4& a, const u32x4& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// 16-byte chunk c of row r of a tile is turned about, so that the four rows of
// two chunks, or the eight of one, that an instruction reads at once lie in
// different banks.
__device__ __forceinline__ constexpr int turn(int r) { return (r & 3) << 1 | (r >> 2 & 1); }
template <int CHUNKS>
__device__ __forceinline__ int place(int r, int c) {
  return (r * CHUNKS + (c ^ turn(r))) * 16;
}

// Half an operand from a tile of 16-bit elements, transposed: the lane's column of
// four rows, of which every lane of 16 addresses four columns of one.
__device__ __forceinline__ uint2 transposed(const uint8_t* p) {
  return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p));
}

// a and b as two bf16 numbers each, to 2^-15: their upper halves, and what those leave, rounded.
// 2048 tokens of 160 heads take 94.4 us so, 95.0 with the upper ones rounded too (2^-16), 91.9 with
// none (2^-14, and always towards zero).
__device__ __forceinline__ void split2(float a, float b, uint32_t& upper, uint32_t& lower) {
  upper = __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
  lower = pack_bf16(a - bf16_hi(__float_as_uint(a)), b - bf16_hi(__float_as_uint(b)));
}

// v exactly, as three numbers of 8 bits: what its upper half holds, what the
// upper half of the rest holds, and the rest.
__device__ __forceinline__ void split3(const float (&v)[8], u32x4 (&part)[3]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a = v[2 * i], b = v[2 * i + 1];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      part[k][i] = __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
      a -= bf16_hi(__float_as_uint(a)), b -= bf16_hi(__float_as_uint(b));
    }
  }
}

// v of another lane of the row of 16 (or of the wave), 0 where there is none.
template <int CTRL>
__device__ __forceinline__ float moved(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float of_lane(float v, int lane) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), lane));
}
// Sums of the lane's and all earlier (later) lanes of its half of the wave.
__device__ __forceinline__ float sums_up(float v, int lane) {
  v += moved<0x111>(v), v += moved<0x112>(v), v += moved<0x114>(v), v += moved<0x118>(v);  // row_shr
  const float a = of_lane(v, 15), b = of_lane(v, 47);
  return v + (lane & 16 ? lane & 32 ? b : a : 0.f);
}
__device__ __forceinline__ float sums_down(float v, int lane) {
  v += moved<0x101>(v), v += moved<0x102>(v), v += moved<0x104>(v), v += moved<0x108>(v);  // row_shl
  const float a = of_lane(v, 16), b = of_lane(v, 48);
  return v + (lane & 16 ? 0.f : lane & 32 ? b : a);
}

// What the first launch leaves for a block of a head, in the order of operands' lanes, 1 KB
// each: M^T of the rows s < 16, whose t < 16 alone are not zero: the bf16 numbers in the
// first half of k, what they leave in the second; M^T of the other rows; what that
// leaves. Then exp(L) and exp(L[31] - L) D of its tokens.
constexpr int kHeadBytes = kScanHeadBytes, kFactors = 3 * 1024;
static_assert(kHeadBytes == kFactors + 2 * kBlock * 4, "layout of a head's block");

// Place of a block in the workspace: blocks of a sequence start at its rows
// begin + 32 i, so row / 32 + s differs for all of them.
__device__ __forceinline__ int64_t block_at(int64_t row, int s) { return (row >> 5) + s; }

// M and factors: a workgroup takes a block of a sequence and eight heads of a
// group, two a wave. Its first three waves make C B^T, 16 x 16 blocks each. Bound
// by the chain of loads, sums and products of each workgroup, then by writing M, 3 KB a
// head and block.
template <int N>
__global__ void __launch_bounds__(256) tern_scan_prepare_kernel(ScanArgs a, uint8_t* ws) {
  __shared__ __attribute__((aligned(16))) f32x4 blocks[3][64];
  __shared__ __attribute__((aligned(16))) float shared[4][2][2][kBlock];  // L and D of a wave's heads
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, low = lane & 31, half = lane >> 5;
  const int low16 = lane & 15, quarter = lane >> 4;
  const int hpg = a.heads / a.groups, parts = (hpg + kScanPrepareHeads - 1) / kScanPrepareHeads;
  const int count = (a.batch.max_q + kBlock - 1) / kBlock;
  int at = blockIdx.x;
  const int h0 = at % parts * kScanPrepareHeads + 2 * wave;  // of the group
  at /= parts;
  const int g = at % a.groups;
  at /= a.groups;
  const int s = at / count, t0 = (at - s * count) * kBlock;
  const Rows rows = rows_of(a.batch, s);
  if (t0 >= rows.n) return;
  const int last = min(rows.n - t0, kBlock);
  const int64_t row0 = rows.row + t0;
  // a token a lane, a head each half
  const int h = g * hpg + min(h0 + half, hpg - 1);
  const int64_t step = (row0 + min(low, last - 1)) * a.dt_stride + h;
  float D = a.dt_type == TERN_F32 ? ((const float*)a.dt)[step] : __uint_as_float((uint32_t)((const uint16_t*)a.dt)[step] << 16);
  const float rate = a.a[h] * kLog2e, bias = a.dt_bias ? a.dt_bias[h] : 0.f;
  // C B^T of the block, transposed, in 16 x 16 blocks (t, s): (0, 0), (0, 1), (1, 1)
  if (wave < 3) {
    const uint16_t* b = a.b + (row0 + min(wave == 2 ? 16 + low16 : low16, last - 1)) * a.b_stride + g * N + 8 * quarter;
    const uint16_t* c = a.c + (row0 + min(wave == 0 ? low16 : 16 + low16, last - 1)) * a.c_stride + g * N + 8 * quarter;
    u32x4 bf[N / 32], cf[N / 32];
#pragma unroll
    for (int q = 0; q < N / 32; ++q) bf[q] = *(const u32x4*)(b + 32 * q), cf[q] = *(const u32x4*)(c + 32 * q);
    f32x4 cb{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int q = 0; q < N / 32; ++q) cb = mfma(bf[q], cf[q], cb);
    blocks[wave][lane] = cb;
  }
  D += bias;
  if (a.softplus) D = softplus(D);
  float e = D * rate;
  e = e < -216.f ? -216.f : e;  // 2^-216 is 0 in fp32; a longer sum would only lose bits of the others
  if (low >= last) D = 0.f, e = 0.f;
  const float L = sums_up(e, lane), R = sums_down(e, lane);
  const float next = moved<0x130>(R);  // wave_shl: the next lane's, the sum behind the token
  const float behind = low == 31 ? 0.f : next;
  shared[wave][half][0][low] = L, shared[wave][half][1][low] = D;
  if (h0 + half < hpg) {
    float* to = (float*)(ws + (block_at(row0, s) * a.heads + h) * kHeadBytes + kFactors) + low;
    to[0] = __builtin_amdgcn_exp2f(L), to[kBlock] = D * __builtin_amdgcn_exp2f(behind);
  }
  __syncthreads();
  const int over = low16 - 4 * quarter;  // s - t + k in the blocks on the diagonal
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (h0 + i >= hpg) break;
    const float(&Ls)[kBlock] = shared[wave][i][0];
    const float(&Ds)[kBlock] = shared[wave][i][1];
    const float own[2] = {Ls[low16], Ls[16 + low16]};
    uint2 out[3], left[3];
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      const int t = j == 2 ? 16 : 0;
      const f32x4 cb = blocks[j][lane], ft = *(const f32x4*)&Ls[t + 4 * quarter], fd = *(const f32x4*)&Ds[t + 4 * quarter];
      float m[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        m[k] = cb[k] * (__builtin_amdgcn_exp2f(own[j > 0] - ft[k]) * fd[k]);
        if (j != 1) m[k] = over < k ? 0.f : m[k];
      }
      split2(m[0], m[1], out[j].x, left[j].x), split2(m[2], m[3], out[j].y, left[j].y);
    }
    u32x4* to = (u32x4*)(ws + (block_at(row0, s) * a.heads + g * hpg + h0 + i) * kHeadBytes) + lane;
    to[0] = u32x4{out[0].x, out[0].y, left[0].x, left[0].y};
    to[64] = u32x4{out[1].x, out[1].y, out[2].x, out[2].y};
    to[128] = u32x4{left[1].x, left[1].y, left[2].x, left[2].y};
  }
}

// Where the state at the start of segment j of a unit lies, for strip 0 of it: states in
// the order of the registers, [N / 16][lane] times four, behind them one decay a strip,
// that of the segment before, as a fraction and a power of two.
__device__ __forceinline__ int64_t state_at(int unit, int units, int j) { return ((int64_t)j * units + unit) * 4; }

template <int P, int N, bool STATES>
__global__ void __launch_bounds__(512, N == 256 ? 2 : 4) tern_scan_blocks_kernel(ScanArgs a, ScanPlan plan, const uint8_t* prepared, float* ws) {
  constexpr int HEADS = P == 32 ? 2 : 1;           // of a workgroup
  constexpr int NB = N / 32, KQ = N / 64, CH = N / 8;  // of a wave: 16-row blocks of the state, steps of 32; chunks of a row of B
  constexpr int ROW = CH * 16;                     // bytes
  constexpr int BL = (kBlock * CH + 511) / 512, BR = 512 / CH;  // chunks a thread copies, rows apart
  __shared__ __attribute__((aligned(16))) uint8_t xs[2][kBlock * 128];  // tiles of blocks in turn
  __shared__ __attribute__((aligned(16))) uint8_t bs[2][kBlock * ROW];
  __shared__ __attribute__((aligned(16))) uint8_t cs[2][STATES ? 16 : kBlock * ROW];
  __shared__ __attribute__((aligned(16))) float fs[2][8][2 * kBlock];  // each wave's factors
  __shared__ __attribute__((aligned(16))) f32x4 parts[2][STATES ? 1 : 8][64];  // of y, for the other half's wave
  __shared__ __attribute__((aligned(16))) uint8_t ys[STATES ? 16 : 8 * 16 * 40];  // 16 rows of 16 columns of y a wave

  // Consecutive workgroups go to the eight dies in turn; neighbours in this order,
  // which share B and C, go to one die.
  const int per = gridDim.x >> 3, rest = gridDim.x & 7, die = blockIdx.x & 7;
  int at = die * per + min(die, rest) + (blockIdx.x >> 3);
  const int hpg = a.heads / a.groups, tiles = (hpg * P + 63) / 64;
  const int units = tiles * a.groups * a.batch.seqs;
  const int seg = at / units, unit = at - seg * units;
  at = unit;
  const int tile = at % tiles;
  at /= tiles;
  const int g = at % a.groups, s = at / a.groups;
  const Rows rows = rows_of(a.batch, s);
  const int first = seg * plan.length;
  if (first >= rows.n) return;
  const int last = min(rows.n - first, plan.length);  // tokens of this segment
  const bool ends = first + last == rows.n;
  if (STATES && ends) return;  // nobody starts from it

  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int strip = wave & 3, upper = wave >> 2;  // 16 columns of x; half of the state's rows
  const int low = lane & 15, quarter = lane >> 4;
  const int head0 = g * hpg + tile * 64 / P, held = min(HEADS, hpg - tile * 64 / P);
  const int hd = strip * 16 / P % HEADS;
  const bool live = hd < held;
  const int head = head0 + min(hd, held - 1);
  const int column = (tile * 64 + strip * 16) % P;  // the strip's first in its head
  const int columns = min(64, hpg * P - tile * 64);
  const int64_t row0 = rows.row + first;
  const int xstep = (int)a.x_stride * 2, bstep = (int)a.b_stride * 2, cstep = (int)a.c_stride * 2, ystep = a.heads * P * 2;

  // ---- copies of a block's rows: global to registers (rows behind the last one
  // are past the end of the resource and read as zeros), registers to LDS.
  const bool copies_x = tid < kBlock * 8, copies_b = kBlock * CH >= 512 || tid < kBlock * CH;
  const int xoff = copies_x && tid % 8 * 8 < columns ? tid / 8 * xstep + tid % 8 * 16 : kOffPastEnd;
  const int brow = tid / CH, bch = tid % CH;
  const int boff = copies_b ? brow * bstep + bch * 16 : kOffPastEnd, coff = copies_b ? brow * cstep + bch * 16 : kOffPastEnd;
  const uint16_t* x = a.x + row0 * a.x_stride + (int64_t)g * hpg * P + tile * 64;
  const uint16_t* b = a.b + row0 * a.b_stride + g * N;
  const uint16_t* c = a.c + row0 * a.c_stride + g * N;
  const uint8_t* from = prepared + (block_at(row0, s) * a.heads + head) * kHeadBytes;
  const int64_t next = (int64_t)a.heads * kHeadBytes;
  struct {  // the block on its way
    u32x4 x, b[BL], c[STATES ? 1 : BL];
    float f;
  } ahead;
  u32x4 m, m_left;  // M^T of the wave's rows s, of the block worked on next
  const int moff = 1024 * upper + 16 * lane, mleft = upper ? 2048 + 16 * lane : kOffPastEnd;
  const uint8_t* from_m = from;
  auto ask_m = [&](bool in) {
    const rsrc_t pres = make_rsrc(from_m, in ? kHeadBytes : 0);
    m = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(pres, moff, 0, 0));
    m_left = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(pres, mleft, 0, 0));
  };
  // Behind the last block every load is past the end, and costs nothing.
  auto ask = [&](int t0) {
    const int n = min(last - t0, kBlock) - 1;
    const bool in = n >= 0;
    const rsrc_t xres = make_rsrc(x, in ? n * xstep + columns * 2 : 0);
    const rsrc_t bres = make_rsrc(b, in ? n * bstep + 2 * N : 0);
    const rsrc_t pres = make_rsrc(from, in ? kHeadBytes : 0);
    ahead.x = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(xres, xoff, 0, 0));
#pragma unroll
    for (int i = 0; i < BL; ++i)
      ahead.b[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(bres, boff + BR * i * bstep, 0, 0));
    ahead.f = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(pres, kFactors + 4 * lane, 0, 0));
    if constexpr (!STATES) {
      const rsrc_t cres = make_rsrc(c, in ? n * cstep + 2 * N : 0);
#pragma unroll
      for (int i = 0; i < BL; ++i)
        ahead.c[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(cres, coff + BR * i * cstep, 0, 0));
      c += kBlock * a.c_stride;
    }
    x += kBlock * a.x_stride, b += kBlock * a.b_stride, from += next;
  };
  // C's chunks hold the k of a quarter wave: columns 4 q .. 4 q + 3 and 16 + 4 q .. of every 32.
  static_assert(BR % 8 == 0, "a thread's rows are turned alike");
  const int xput = place<8>(tid / 8, tid % 8), bput = place<CH>(brow, bch);
  const int cput = place<CH>(brow, (bch & ~3) + (bch & 1) * 2) + (bch >> 1 & 1) * 8;
  const int cput1 = place<CH>(brow, (bch & ~3) + (bch & 1) * 2 + 1) + (bch >> 1 & 1) * 8;
  float total;  // the decay of the block whose tiles were put last
  auto put = [&](int turn) {
    if (copies_x) *(u32x4*)(xs[turn] + xput) = ahead.x;
    if (copies_b) {
#pragma unroll
      for (int i = 0; i < BL; ++i) {
        *(u32x4*)(bs[turn] + bput + BR * i * ROW) = ahead.b[i];
        if constexpr (!STATES) {
          *(uint2*)(cs[turn] + cput + BR * i * ROW) = uint2{ahead.c[i][0], ahead.c[i][1]};
          *(uint2*)(cs[turn] + cput1 + BR * i * ROW) = uint2{ahead.c[i][2], ahead.c[i][3]};
        }
      }
    }
    fs[turn][wave][lane] = ahead.f;
    total = of_lane(ahead.f, 31);
  };
  ask(0);
  if constexpr (!STATES) ask_m(true);

  // ---- the state at the segment's start: register r of block nb holds row
  // 16 nb + 4 quarter + r of the wave's half
  f32x4 S[NB];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) S[nb] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int64_t mine = ((int64_t)head * N + upper * (N / 2)) * P + column;  // of the wave
  const int64_t slot = (int64_t)a.heads * N * P;
  constexpr int64_t kWave = N * 16;
  if constexpr (!STATES) {
    // The first segment's too, if there are others: the slot may be the one that the last of
    // them writes in this launch.
    if (!(seg == 0 && ends)) {
      const f32x4* p = (const f32x4*)(ws + (state_at(unit, units, seg) + strip) * kWave) + upper * NB * 64 + lane;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) S[nb] = p[nb * 64];
    } else {
      const int src = a.batch.src[s];
      if (src >= 0 && src < a.slots) {
        const float* p = a.state + src * slot + mine + 4 * quarter * P + low;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int r = 0; r < 4; ++r) S[nb][r] = p[(16 * nb + r) * P];
      }
    }
  }
  // The segment's decay, fraction 2^power: where states grow, the product of its blocks'
  // factors may leave fp32 though none of them does and no state.
  float fraction = 1.f;
  int power = 0;

  // ---- what a lane reads of the tiles; the rest of an address is constant
  const int tr = 4 * quarter + (lane >> 2 & 3), piece = lane & 3;  // transposed: row, 4 columns
  const int xt = place<8>(tr, 2 * strip + (piece >> 1)) + (piece & 1) * 8;
  constexpr int BT = NB < 4 ? NB : 4, CO = KQ < 2 ? KQ : 2;
  int bt[BT], co[2][CO];  // C's rows that the wave ends, and the other wave's
#pragma unroll
  for (int i = 0; i < BT; ++i) bt[i] = place<CH>(tr, 2 * (upper * NB + i) + (piece >> 1)) + (piece & 1) * 8;
#pragma unroll
  for (int i = 0; i < CO; ++i) {
    co[0][i] = place<CH>(16 * upper + low, 4 * (upper * KQ + i) + quarter);
    co[1][i] = place<CH>(16 - 16 * upper + low, 4 * (upper * KQ + i) + quarter);
  }

  // y of a block leaves while the next one is worked on: the wave of each half of
  // the state ends 16 of its rows, with the other's part of them, and brings them through
  // its own part of LDS to whole 32-byte pieces.
  uint8_t* const yput = ys + (STATES ? 0 : wave * 16 * 40 + low * 40 + quarter * 8);
  const uint8_t* const yget = ys + (STATES ? 0 : wave * 16 * 40 + (lane >> 2) * 40 + (lane & 3) * 8);
  const int yoff = (16 * upper + (lane >> 2)) * ystep + 2 * column + (lane & 3) * 8;
  uint16_t* y = a.y + (row0 * a.heads + head) * P;
  const float skip = a.d ? a.d[head] : 0.f;
  const int xown = place<8>(16 * upper + low, 2 * strip + (quarter >> 1)) + (quarter & 1) * 8;
  f32x4 out{0.f, 0.f, 0.f, 0.f};
  float scale = 0.f;  // exp(L) of the lane's row
  auto store_y = [&](const f32x4& out, float scale, int t0, int turn) {  // of block t0
    const f32x4 other = parts[turn][wave ^ 4][lane];
    float v[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = __builtin_fmaf(scale, other[r], out[r]);
    *(uint2*)yput = uint2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    const int n = min(last - t0, kBlock) - 1;
    const rsrc_t yres = make_rsrc(y + (int64_t)t0 * a.heads * P, live ? n * ystep + 2 * P : 0);
    typedef int i32x2 __attribute__((ext_vector_type(2)));
    __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(i32x2, *(const uint2*)yget), yres, yoff, 0, 0);
  };

  // Block t0, whose tiles lie in buffer `turn`. The next one's go into the other
  // buffer, which was read before the last barrier.
  auto step = [&](auto constant, int t0) {
    constexpr int turn = decltype(constant)::value;
    const float factor = total;
    const uint2 x0 = transposed(xs[turn] + xt), x1 = transposed(xs[turn] + xt + 16 * 128);
    const u32x4 xf{x0.x, x0.y, x1.x, x1.y};  // x^T of the strip
    const f32x4 before = out;
    const float before_scale = scale;
    // ---- the half's part of y^T = S^T C^T, scaled; x^T M^T for the wave's rows
    f32x4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    if constexpr (!STATES) {
      u32x4 high[KQ], lower[KQ];
#pragma unroll
      for (int q = 0; q < KQ; ++q)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t h, l;
          split2(S[2 * q + (j >> 1)][2 * (j & 1)], S[2 * q + (j >> 1)][2 * (j & 1) + 1], h, l);
          high[q][j] = h, lower[q][j] = l;
        }
#pragma unroll
      for (int q = 0; q < KQ; ++q)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const u32x4 ct = *(const u32x4*)(cs[turn] + co[j][q & 1] + (q >> 1) * 128);
          acc[j] = mfma(high[q], ct, acc[j]);
          acc[j] = mfma(lower[q], ct, acc[j]);
        }
      parts[turn][wave][lane] = acc[1];
      scale = fs[turn][wave][16 * upper + low];
      const uint2 own = *(const uint2*)(xs[turn] + xown);
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[0][r] *= scale;
      acc[0][0] = __builtin_fmaf(skip, bf16_lo(own.x), acc[0][0]), acc[0][1] = __builtin_fmaf(skip, bf16_hi(own.x), acc[0][1]);
      acc[0][2] = __builtin_fmaf(skip, bf16_lo(own.y), acc[0][2]), acc[0][3] = __builtin_fmaf(skip, bf16_hi(own.y), acc[0][3]);
      // the rows s < 16 meet the rows t < 16 twice, with M and with what it left
      out = mfma(xf, m_left, mfma(upper ? xf : u32x4{xf[0], xf[1], xf[0], xf[1]}, m, acc[0]));
      from_m += next;
      ask_m(t0 + kBlock < last);
    }
    // The next block's copies wait until this one's operands of y are read: in front of them they
    // take 151 and not 144 us of 2048 tokens of 160 heads of 128 x 128, 145 and 141 of 64 x 256, 96 and 95
    // of 64 x 128; 81.0 and 81.2 of 64 x 64, and a microsecond less where a call has 16 blocks.
    put(turn ^ 1), ask(t0 + 2 * kBlock);
    // ---- the next state
    if constexpr (STATES) {
      fraction *= __builtin_amdgcn_frexp_mantf(factor);
      power += __builtin_amdgcn_frexp_expf(factor) + __builtin_amdgcn_frexp_expf(fraction);
      fraction = __builtin_amdgcn_frexp_mantf(fraction);
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int r = 0; r < 4; ++r) S[nb][r] *= factor;
    {
      float v[8];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const f32x4 w = *(const f32x4*)&fs[turn][wave][kBlock + 16 * j + 4 * quarter];
        v[4 * j] = w[0] * bf16_lo(xf[2 * j]), v[4 * j + 1] = w[1] * bf16_hi(xf[2 * j]);
        v[4 * j + 2] = w[2] * bf16_lo(xf[2 * j + 1]), v[4 * j + 3] = w[3] * bf16_hi(xf[2 * j + 1]);
      }
      u32x4 part[3];
      split3(v, part);
#pragma unroll
      for (int n4 = 0; n4 < NB; n4 += BT) {
        u32x4 bf[BT];
#pragma unroll
        for (int i = 0; i < BT; ++i) {
          const uint8_t* p = bs[turn] + bt[i] + (n4 >> 2) * 128;
          const uint2 lo = transposed(p), hi = transposed(p + 16 * ROW);
          bf[i] = u32x4{lo.x, lo.y, hi.x, hi.y};
        }
#pragma unroll
        for (int k = 0; k < 3; ++k)
#pragma unroll
          for (int i = 0; i < BT; ++i) S[n4 + i] = mfma(bf[i], part[k], S[n4 + i]);
      }
    }
    if constexpr (!STATES) {
      if (t0 > 0) store_y(before, before_scale, t0 - kBlock, turn ^ 1);
      // A value of x that is not finite has reached the rows before it, through
      // zeros of M: the product is made again without it, and its column's results
      // from its row on are NaN.
      u16x2 top = {0, 0};
#pragma unroll
      for (int i = 0; i < 4; ++i) top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, xf[i] & 0x7fff7fffu));
      if (__any(max((uint32_t)top.x, (uint32_t)top.y) >= 0x7f80u)) {
        u32x4 clean = xf;
        int at = 8;  // the lane's first, in the order of its rows
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t w = xf[i >> 1] >> (16 * (i & 1));
          if ((w & 0x7f80u) == 0x7f80u) {
            at = min(at, i);
            clean[i >> 1] &= i & 1 ? 0xffffu : 0xffff0000u;
          }
        }
        int bad = at == 8 ? kBlock : (at >> 2) * 16 + 4 * quarter + (at & 3);
        bad = min(bad, __shfl_xor(bad, 16));
        bad = min(bad, __shfl_xor(bad, 32));
        from_m -= next;
        ask_m(true);
        out = mfma(clean, m_left, mfma(upper ? clean : u32x4{clean[0], clean[1], clean[0], clean[1]}, m, acc[0]));
        from_m += next;
        ask_m(t0 + kBlock < last);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int since = __shfl(bad, 4 * quarter + r);
          if (16 * upper + low >= since) out[r] = __builtin_nanf("");
        }
      }
    }
    __syncthreads();
  };
  put(0);
  ask(kBlock);
  __syncthreads();
  int t0 = 0, turn = 0;
  for (;;) {
    step(std::integral_constant<int, 0>{}, t0);
    turn = 0;
    if ((t0 += kBlock) >= last) break;
    step(std::integral_constant<int, 1>{}, t0);
    turn = 1;
    if ((t0 += kBlock) >= last) break;
  }
  if constexpr (!STATES) store_y(out, scale, t0 - kBlock, turn);
  if constexpr (STATES) {
    const int64_t to = state_at(unit, units, seg + 1) + strip;
    f32x4* p = (f32x4*)(ws + to * kWave) + upper * NB * 64 + lane;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) p[nb * 64] = S[nb];
    if (lane == 0 && !upper)
      *(float2*)(ws + state_at(0, units, plan.segments) * kWave + 2 * to) = float2{fraction, __int_as_float(power)};
  } else {
    const int dst = a.batch.dst[s];
    if (ends && live && dst >= 0 && dst < a.slots) {
      // the lane's number anew: kept, its place would be in memory through the loop
      const int l = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0));
      float* p = a.state + dst * slot + mine + 4 * (l >> 4) * P + (l & 15);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int r = 0; r < 4; ++r) p[(16 * nb + r) * P] = S[nb][r];
    }
  }
}

// Turns the segments' own states into the states at the segments' starts: state 0 is
// the sequence's, state j becomes decay_j (the one before it) + state j. A thread
// takes four elements of a strip's state through all segments, whose loads go out
// eight at a time.
template <int P, int N>
__global__ void __launch_bounds__(256) tern_scan_join_kernel(ScanArgs a, ScanPlan plan, float* ws) {
  constexpr int HEADS = P == 32 ? 2 : 1, NB = N / 16, AT_ONCE = 8;
  constexpr int64_t kWave = N * 16;
  const int hpg = a.heads / a.groups, tiles = (hpg * P + 63) / 64;
  const int units = tiles * a.groups * a.batch.seqs;
  const int lane = threadIdx.x & 63, quarter = lane >> 4, low = lane & 15;
  const int64_t piece = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);  // 16 rows of a wave's state
  const int nb = (int)(piece % NB), wave = (int)(piece / NB % 4), unit = (int)(piece / (4 * NB));
  const int tile = unit % tiles, g = unit / tiles % a.groups, s = unit / (tiles * a.groups);
  const Rows rows = rows_of(a.batch, s);
  const int count = rows.n == 0 ? 0 : (rows.n - 1) / plan.length;  // segments that another starts from
  if (count == 0) return;
  const int head0 = g * hpg + tile * 64 / P, held = min(HEADS, hpg - tile * 64 / P);
  const int head = head0 + min(wave * 16 / P % HEADS, held - 1), column = (tile * 64 + wave * 16) % P;
  f32x4 S{0.f, 0.f, 0.f, 0.f};
  const int src = a.batch.src[s];
  if (src >= 0 && src < a.slots) {
    const float* p = a.state + ((int64_t)src * a.heads + head) * N * P + (16 * nb + 4 * quarter) * P + column + low;
#pragma unroll
    for (int r = 0; r < 4; ++r) S[r] = p[r * P];
  }
  const float2* decays = (const float2*)(ws + state_at(0, units, plan.segments) * kWave);
  f32x4* at = (f32x4*)(ws + (state_at(unit, units, 0) + wave) * kWave) + nb * 64 + lane;
  const int64_t step = (int64_t)units * kWave;  // of four floats: a segment
  at[0] = S;
  for (int j0 = 1; j0 <= count; j0 += AT_ONCE) {
    f32x4 v[AT_ONCE];
    float2 decay[AT_ONCE];
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) {
      const int j = min(j0 + i, count);
      v[i] = at[j * step], decay[i] = decays[state_at(unit, units, j) + wave];
    }
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) {
      if (j0 + i > count) break;
#pragma unroll
      for (int r = 0; r < 4; ++r) S[r] = __builtin_ldexpf(S[r] * decay[i].x, __float_as_int(decay[i].y)) + v[i][r];
      at[(j0 + i) * step] = S;
    }
  }
}

template <int N>
int go_prepare(const ScanArgs& a, uint8_t* prepared, hipStream_t st) {
  tern_scan_prepare_kernel<N><<<dim3((unsigned)scan_prepare_blocks(a)), dim3(256), 0, st>>>(a, prepared);
  return kernel_launched((int)hipGetLastError(), TERN_KERNEL_SCAN_PREPARE);
}

template <int P, int N>
int go(const ScanArgs& a, const ScanPlan& p, uint8_t* ws, hipStream_t st) {
  if (int err = go_prepare<N>(a, ws, st)) return err;
  float* states = (float*)(ws + scan_prepared_bytes(a));
  const int64_t units = scan_units(a);
  if (p.segments > 1) {
    tern_scan_blocks_kernel<P, N, true><<<dim3((unsigned)(units * (p.segments - 1))), dim3(512), 0, st>>>(a, p, ws, states);
    if (int err = kernel_launched((int)hipGetLastError(), TERN_KERNEL_SCAN_STATES)) return err;
    tern_scan_join_kernel<P, N><<<dim3((unsigned)(units * (N / 16))), dim3(256), 0, st>>>(a, p, states);
    if (int err = kernel_launched((int)hipGetLastError(), TERN_KERNEL_SCAN_JOIN)) return err;
  }
  tern_scan_blocks_kernel<P, N, false><<<dim3((unsigned)(units * p.segments)), dim3(512), 0, st>>>(a, p, ws, states);
  return kernel_launched((int)hipGetLastError(), TERN_KERNEL_SCAN_BLOCKS);
}

template <int P>
int go_p(const ScanArgs& a, const ScanPlan& p, uint8_t* ws, hipStream_t st) {
  if (a.state_dim == 64) return go<P, 64>(a, p, ws, st);
  if (a.state_dim == 128) return go<P, 128>(a, p, ws, st);
  return go<P, 256>(a, p, ws, st);
}

}  // namespace

int launch_scan_blocks(const ScanArgs& a, const ScanPlan& p, void* ws, void* stream) {
  hipStream_t st = (hipStream_t)stream;
  if (a.dim == 32) return go_p<32>(a, p, (uint8_t*)ws, st);
  if (a.dim == 64) return go_p<64>(a, p, (uint8_t*)ws, st);
  return go_p<128>(a, p, (uint8_t*)ws, st);
}

}  // namespace tern
