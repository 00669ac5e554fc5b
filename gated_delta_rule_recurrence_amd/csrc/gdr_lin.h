// The chunked form of linear attention (formulas in gdr_lin.hip): tiles of L
// steps of one head, their products on matrix cores.
//
// With H_r the summed log decays up to row r of a tile (its own included; for
// dk and dv, whose tiles hold the steps in reverse, only those of the rows
// before), P_ij = scale exp(H_i - H_j) Q_i.K_j for j <= i:
//   out_i = sum_j P_ij V_j + cf_i S Q_i,          cf_i = exp(H_i)
//   S <- exp(total) S + sum_j uf_j V_j K_j^T,     uf_j = exp(total - H_j)
// H is summed and subtracted in 64 bits: a difference of two of them keeps the
// accuracy of the few steps between, however much the tile has decayed.  A log
// decay below kLeastLog counts as that, so that -inf forgets without a
// difference of infinities; a segment that holds one keeps nothing of its state.
//
// Decays that grow.  Where the positive ones of a tile sum to more than kGrows,
// factors that the recurrence never forms alone (exp(H_i), P_ij) could pass
// fp32's range while what they multiply is small or 0.  Such a tile is walked in
// passes, each over the rows [x0, x1) that grow by no more (lin_pass); a step
// that grows by more alone is a pass of the state only, or several.  (What the
// other tiles pay for it: 0 to 1% of a pass, 5% of the small fp32 one, 86 us.)
//
// Precision.  bf16 rows are matrix operands as they are; what is fp32 (P, S,
// uf V) enters a product in three bf16 pieces, which hold fp32's 24 bits.  (Two
// hold 18: enough for a bf16 output by itself, but not where large terms cancel
// in it.  Seven prompts 154 us with two and 163 with three, training of 2048
// steps, heads 16/64 of 192/128, 468 and 480, 4 x 4096 steps of 32 heads of
// 128/128 760 and 843; the bf16 outputs' difference to a plain fp32 form 1.0e-4
// and 0.4e-4.)  fp32 rows are three pieces too; of the nine products the six
// above 2^-24 are formed (with the next two the errors are the same).
//
// Mapping.  A workgroup of four waves runs through a segment of one sequence
// for one head and NT 64 columns of its output.  P is formed by all waves, in
// LDS; each wave then owns 16 NT columns of out and of the state, which stays
// in its registers: an accumulator's layout (lane l: row 4 (l / 16) + v, column
// l % 16) is an operand's (lane l: index l % 16, k = 8 (l / 16) + e) where two
// accumulators' rows are dealt to the lanes in turn, so the update's left
// operand is read from LDS in that order and the state needs no exchange.  Out
// is formed transposed, so that a lane holds four neighbouring columns of one
// row.
//
// What bounds it: the dependent phases of a tile (P, S Q, P's decays, P V and the
// update, with three barriers) at the two waves a SIMD that the state leaves
// registers for.  4 x 4096 steps of 32 heads of 128/128: states alone 92 us, y
// 195, dq with dk and dv 534 to 549; there the vector units are 37, 41 and 51%
// busy, matrix cores 23, 30 and 34, LDS 14, 19 and 22, HBM at 2.7 to 3.3 TB/s.
// Eight waves of 16 columns have more to switch between and 47% more vector
// instructions, as each forms the same operands (with operands of two pieces 812
// us a pass against 722).
#pragma once

#include "gdr_layer.h"

namespace gdr {

constexpr int kLinWaves = 4;  // waves of a workgroup
// (what a kLeastLog leaves is 0 after a pass's growth, any value but 0 that grows
// by kMostLog is past fp32's range)
constexpr double kLeastLog = -1000.0, kMostLog = 200.0, kGrows = 40.0;
// An offset past the end of every buffer (64 rows of at most 2^23 elements).
constexpr uint32_t kLinPast = 0xf0000000u;

// One of the four products (gdr_lin.hip).
struct LinRole {
  const void* Q;
  const void* K;
  const void* V;
  const void* R;       // with flow: rows that out's earlier part is multiplied with
  int64_t sq, sk, sv, sr;
  int dq, dk, dv, dr;  // value heads per head of each
  int Ni, No, tiles;   // contracted width, output width, workgroups over it
  float ps, cs, us;    // factors of P, of cf and of uf
  int reverse;         // time runs backwards
  int transposed;      // states lie [Ni][No] instead of [No][Ni]
  int vec;             // widths and strides are whole vectors (VEC)
  const float* first;  // states before each segment, or null (zeros)
  int slots;           // they lie in segments' slots, not [B][Hv]
  float* last;         // [B][Hv] states behind the sequences (one segment), or null
  float* save;         // slots of the state before and behind (one segment), or null
  float* local;        // states only: slots of the segments' own ends
  double* decay;       // states only: [slots][Hv] summed log decays of the segments
  void* out;           // [rows][Hv][No], or null
  float* part;         // the same in fp32
  float* flow;         // [tiles][Hv][rows]: R out, without the step's own term
};

enum LinMode { kLinOut = 0, kLinFlow = 1, kLinState = 2 };

// Slot of segment s of sequence b: sequences own more slots than segments, for
// the state behind the last.  One of no rows owns none and writes none: it may
// stand anywhere, so its slots here may be another's.
__device__ __forceinline__ int64_t lin_slot(const LinArgs& a, Span sp, int b, int s) {
  return sp.first / a.seg + 2 * (int64_t)b + s;
}

__device__ __forceinline__ float lin_log_decay(const LinArgs& a, int64_t row, int h) {
  if (a.log_g == nullptr) return 0.f;
  const int64_t at = a.per_head ? h : row * a.g_stride + h;
  return a.g_bf16 ? to_f32(static_cast<const bf16*>(a.log_g)[at])
                  : static_cast<const float*>(a.log_g)[at];
}

template <typename T>
struct LinTypes;
template <>
struct LinTypes<bf16> {
  static constexpr int L = 64, NP = 1;
};
template <>
struct LinTypes<float> {
  static constexpr int L = 32, NP = 3;
};
constexpr int kLinPieces = 3;  // of an fp32 operand

// A tile [rows][W] of bf16 in LDS whose 16-byte blocks are exchanged inside a
// row, block ^ lin_swz(row).  The 64 banks hold 16 blocks; what reads them at
// once, as measured: a read by rows 16 lanes, rows 0 .. 3 and 12 .. 15 of one
// block and rows 4 .. 11 of its neighbour (or the others); a transposed read 32
// lanes, rows 0 .. 3 and 8 .. 11 (or the others), two blocks each.  So the bits
// of r but r2 choose the pair of blocks, and r2 and r3 together, which keep
// those two groups of rows apart, the one of it.  (The state's order reads
// halves of four blocks: two cycles for one.)  Conflicts were 42% of the LDS
// cycles with an order that served consecutive rows only.
template <int W>
__device__ __forceinline__ int lin_swz(int r) {
  const int low = ((r & 2) << 1) | (((r >> 2) ^ (r >> 1)) & 2) | ((r >> 2) & 1);
  if constexpr (W % 128 == 0) return ((r & 1) << 3) | low;  // (else r0 is half of the banks)
  if constexpr (W == 32) return low & 3;
  return low;
}
// Element c of row r, where c is a whole block's first for a lane's own `at`
// of another column of the same row: blocks of one row differ by an exclusive
// or, so that a lane forms one place for all reads of a tile and each costs at
// most one more instruction (formed one by one, they were a sixth of all).
template <int W>
__device__ __forceinline__ int lin_move(int at, int c) {
  constexpr int kMask = W % 128 == 0 ? 127 : W == 32 ? 31 : 63;
  return (at ^ (c & kMask)) + (c & ~kMask);
}
// Row r, column c.
template <int W>
__device__ __forceinline__ int lin_at(int r, int c) {
  return lin_move<W>(r * W + (lin_swz<W>(r) << 3), c);
}
// Lane l: row l % 16, columns 8 (l / 16) ..; an operand is read r0 rows (a
// multiple of 16) and c0 columns (of 32) on.
template <int W>
__device__ __forceinline__ int lin_row_place(int lane) {
  return lin_at<W>(lane & 15, 8 * (lane >> 4));
}
template <int W>
__device__ __forceinline__ uint4 lin_rows(const uint16_t* t, int place, int r0, int c0) {
  return *reinterpret_cast<const uint4*>(t + r0 * W + lin_move<W>(place, c0));
}
// Lane l: column l % 16 (STATE: columns 8 (l % 16 / 4) + l % 4), rows
// 8 (l / 16) ..; read r0 rows (of 32) and c0 columns (of 16; STATE: of 32, or 4
// more) on.  The upper four rows' blocks are those of the lower ones ^ 3.
template <int W, bool STATE>
__device__ __forceinline__ int lin_column_place(int lane) {
  return lin_at<W>(8 * (lane >> 4) + ((lane >> 2) & 3), (STATE ? 8 : 4) * (lane & 3));
}
template <int W>
__device__ __forceinline__ uint4 lin_columns(const uint16_t* t, int place, int r0, int c0) {
  const int at = lin_move<W>(place, c0);
  const uint2 lo = lds_read_tr16(t + r0 * W + at);
  const uint2 hi = lds_read_tr16(t + (r0 + 4) * W + (at ^ 24));
  return uint4{lo.x, lo.y, hi.x, hi.y};
}

__device__ __forceinline__ f4 lin_unpack(uint2 w) {
  return f4{__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
            __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u)};
}

// The bf16 pieces of eight values, as operands.
__device__ __forceinline__ void lin_split(f4 a, f4 b, uint4 (&p)[kLinPieces]) {
  uint2 x[3], y[3];
  split3_quad(a, x[0], x[1], x[2]);
  split3_quad(b, y[0], y[1], y[2]);
#pragma unroll
  for (int i = 0; i < kLinPieces; ++i) p[i] = uint4{x[i].x, x[i].y, y[i].x, y[i].y};
}

// c + a b over the pieces' products that fp32 sees.
template <int NA, int NB>
__device__ __forceinline__ f4 lin_mfma(const uint4 (&a)[NA], const uint4 (&b)[NB], f4 c) {
#pragma unroll
  for (int i = NA - 1; i >= 0; --i)
#pragma unroll
    for (int j = NB - 1; j >= 0; --j)
      if (i + j < 3) c = mfma_bf16(a[i], b[j], c);
  return c;
}

// Eight elements of a row as loaded: whole vectors, or elements of which only
// the first n are in the row.
typedef uint16_t LinU16x2 __attribute__((ext_vector_type(2)));
constexpr uint16_t kLinInf = 0x7f80;  // bits of an infinity; those of a NaN are more
template <typename T>
struct LinRaw;
template <>
struct LinRaw<bf16> {
  uint4 v;
  // the largest magnitudes' bits, of even and odd elements
  __device__ __forceinline__ LinU16x2 most(LinU16x2 m) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      m = __builtin_elementwise_max(m, __builtin_bit_cast(LinU16x2, w[i] & 0x7fff7fffu));
    return m;
  }
  __device__ __forceinline__ void put(uint16_t* const (&t)[1], int at) const {
    *reinterpret_cast<uint4*>(t[0] + at) = v;
  }
  __device__ __forceinline__ void load(Buffer p, uint32_t at) {
    v = get_pack<bf16, 8>(p, at).v;
  }
  __device__ __forceinline__ void load(Buffer p, uint32_t at, int n) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = get_pack<bf16, 1>(p, i < n ? at + 2 * i : kLinPast).v[0].bits;
    v = uint4{w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16};
  }
};
template <>
struct LinRaw<float> {
  float4 lo, hi;
  static __device__ __forceinline__ bool finite(float x) {
    return (__float_as_uint(x) >> 16 & 0x7fffu) < kLinInf;
  }
  __device__ __forceinline__ LinU16x2 most(LinU16x2 m) const {
    const float f[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      m = __builtin_elementwise_max(
          m, __builtin_bit_cast(LinU16x2, __float_as_uint(f[i]) >> 16 & 0x7fffu));
    return m;
  }
  __device__ __forceinline__ void put(uint16_t* const (&t)[3], int at) const {
    uint4 p[3];
    f4 a = {lo.x, lo.y, lo.z, lo.w}, b = {hi.x, hi.y, hi.z, hi.w};
    const bool odd = most(LinU16x2{0, 0}).x >= kLinInf;
    if (odd)
      for (int i = 0; i < 4; ++i) {
        a[i] = finite(a[i]) ? a[i] : 0.f;
        b[i] = finite(b[i]) ? b[i] : 0.f;
      }
    lin_split(a, b, p);
#pragma unroll
    for (int i = 0; i < 3; ++i) *reinterpret_cast<uint4*>(t[i] + at) = p[i];
    if (odd) {  // (the split would spoil a neighbour)
      const float f[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (!finite(f[i])) t[0][at + i] = 0x7fff;
    }
  }
  __device__ __forceinline__ void load(Buffer p, uint32_t at) {
    lo = get_pack<float, 4>(p, at).v;
    hi = get_pack<float, 4>(p, at + 16).v;
  }
  __device__ __forceinline__ void load(Buffer p, uint32_t at, int n) {
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = get_pack<float, 1>(p, i < n ? at + 4 * i : kLinPast).v[0];
    lo = float4{w[0], w[1], w[2], w[3]};
    hi = float4{w[4], w[5], w[6], w[7]};
  }
};
// Four elements of a row, of which n are in it, `at` + `more` bytes into p (the
// sum in the offset that the bound is checked with), as loaded.
template <bool VEC, typename T>
struct LinQuad {
  Pack<T, VEC ? 4 : 1> v[VEC ? 1 : 4];
  __device__ __forceinline__ void load(Buffer p, uint32_t at, uint32_t more, int n) {
#pragma unroll
    for (int i = 0; i < (VEC ? 1 : 4); ++i)
      v[i] = get_pack<T, VEC ? 4 : 1>(p, i < n ? at + more + i * sizeof(T) : kLinPast);
  }
  __device__ __forceinline__ f4 get() const {
    float f[4];
    if constexpr (VEC) {
      unpack(v[0], f);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = to_f32(v[i].v[0]);
    }
    return f4{f[0], f[1], f[2], f[3]};
  }
};
template <bool VEC, typename T>
__device__ __forceinline__ void lin_put(Buffer p, uint32_t at, uint32_t more, f4 x, int n) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  if constexpr (VEC) {
    const int to = n > 0 ? at + more : kLinPast;
    if constexpr (sizeof(T) == 2)
      __builtin_amdgcn_raw_buffer_store_b64(
          u32x2{cvt_pk_bf16(x[0], x[1]), cvt_pk_bf16(x[2], x[3])}, p.resource(), to, 0, 0);
    else
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), p.resource(), to,
                                             0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int to = i < n ? at + more + i * sizeof(T) : kLinPast;
      if constexpr (sizeof(T) == 2)
        __builtin_amdgcn_raw_buffer_store_b16((uint16_t)cvt_pk_bf16(x[i], x[i]), p.resource(), to,
                                              0, 0);
      else
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x[i]), p.resource(), to,
                                              0, 0);
    }
  }
}

// Sums over lanes 0 .. l.
template <int CTRL, int ROWS>
__device__ __forceinline__ double lin_dpp(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROWS, 0xF, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, ROWS, 0xF,
                                                  false);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double lin_prefix_sum(double x) {
  x += lin_dpp<0x111, 0xF>(x);  // row_shr:1
  x += lin_dpp<0x112, 0xF>(x);
  x += lin_dpp<0x114, 0xF>(x);
  x += lin_dpp<0x118, 0xF>(x);
  x += lin_dpp<0x142, 0xA>(x);  // row_bcast:15 into rows 1 and 3
  x += lin_dpp<0x143, 0xC>(x);  // row_bcast:31 into rows 2 and 3
  return x;
}

__device__ __forceinline__ float lin_exp(double x) { return exp2_hw(kLog2e * (float)x); }
// s exp(x) where exp(x) may be past fp32's range: 0 stays 0.
__device__ __forceinline__ float lin_grow(float s, double x) {
  const double y = fmin(x * 1.4426950408889634, 1e6);
  const int n = (int)(y - 100.0);
  return ldexpf(s * exp2_hw((float)(y - n)), n);
}

// Where a tile of growing decays is.  Rows behind x1 wait for another pass, and
// the state still has to grow by `debt` before it (`paid`: it has grown by row
// x0's decay).
struct LinPass {
  float debt;
  int x0, paid;
};
constexpr uint32_t lin_part(int x0, int x1, bool done) { return x0 | x1 << 8 | done << 16; }
// The next pass over a tile's log decays x, one a lane of the first L: its part,
// with x as it takes them (0 outside its rows, in lane 0 where the state alone
// grows).  A big step, above kGrows, grows the state before its row's pass, or
// behind it in reverse.  `at` lies in LDS, the same for the whole wave.
template <int L>
__device__ __forceinline__ uint32_t lin_pass(double& x, LinPass& at, bool reverse) {
  const int lane = threadIdx.x & 63, x0 = at.x0;
  x = x > kMostLog ? (x < __builtin_inf() ? kMostLog : __builtin_nan("")) : x;
  x = lane < x0 || (at.paid && lane == x0) ? 0.0 : x;
  const uint64_t big = __ballot(x > kGrows);
  const uint64_t stop = (reverse ? big << 1 : big) |
                        __ballot(lin_prefix_sum(x > 0.0 && x <= kGrows ? x : 0.0) > kGrows);
  float debt = at.debt;
  int x1 = stop != 0 ? __builtin_ctzll(stop) : L;
  x1 = debt > 0.f ? x0 : x1 < L ? x1 : L;
  const int last = reverse ? x1 - 1 : x0;  // the row whose big step is met here
  if (debt == 0.f && (big >> (last & 63) & 1)) debt = __shfl((float)x, last, 64);
  x = lane >= x1 || x > kGrows ? 0.0 : x;
  const bool grow = x1 == x0;  // the state alone
  if (grow) {
    const float by = fminf(debt, 2 * (float)kGrows);
    debt -= by;
    x = lane == 0 ? (double)by : 0.0;
  }
  const bool done = x1 == L && debt == 0.f;
  at = LinPass{debt, done ? 0 : x1, grow && !reverse && debt == 0.f};
  return lin_part(x0, x1, done);
}

// A tile [L][W] on its way through a thread's registers: 8 threads a row,
// eight elements in each 64 columns, 8 kLinWaves rows at a time.
template <typename T, int W>
struct LinStage {
  static constexpr int L = LinTypes<T>::L, NP = LinTypes<T>::NP, R = 8 * kLinWaves;
  static constexpr int NR = L / R, NC = W / 64;
  static_assert(NR * R == L, "whole passes of the threads");
  LinRaw<T> raw[NR][NC];
  // `rows` rows of n columns, `stride` apart, from p on; zeros outside
  template <bool VEC>
  __device__ __forceinline__ void load(const T* p, int64_t stride, int rows, int n, int thread) {
    const Buffer buf = buffer_of(p, 0, (((int64_t)rows - 1) * stride + n) * sizeof(T));
    const int c = (thread & 7) * 8;
    const uint32_t at = ((thread >> 3) * (uint32_t)stride + c) * sizeof(T);
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
      for (int k = 0; k < NC; ++k) {
        const uint32_t to = at + (R * i * (uint32_t)stride + 64 * k) * sizeof(T);
        if constexpr (VEC)
          raw[i][k].load(buf, c + 64 * k < n ? to : kLinPast);
        else
          raw[i][k].load(buf, to, n - c - 64 * k);
      }
  }
  // reverse: the last row first
  __device__ __forceinline__ void store(uint16_t* const (&t)[NP], bool reverse, int thread) const {
    const int x = reverse ? L - 1 - (thread >> 3) : thread >> 3;
    const int at = lin_at<W>(x, (thread & 7) * 8), step = reverse ? -R * W : R * W;
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
      for (int k = 0; k < NC; ++k) raw[i][k].put(t, step * i + lin_move<W>(at, 64 * k));
  }
  // whether one of the elements is not finite
  __device__ __forceinline__ bool odd() const {
    LinU16x2 m = {0, 0};
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
      for (int k = 0; k < NC; ++k) m = raw[i][k].most(m);
    return m.x >= kLinInf || m.y >= kLinInf;
  }
};

// Waves of a SIMD (workgroups of a compute unit) that the registers are cut to,
// no more than LDS holds.  128 contracted columns with 64 of output: three for the
// flows, though some registers are spilled for it (training of 2048 steps, heads
// 16/64 of 192/128, 491 us, with two and no spills 524), two for out alone
// (2 x 2048 steps, heads 1/64 of 128/64, 411 us, with three 422).
template <typename T>
constexpr int lin_waves(int KI, int NT, int MODE) {
  if (sizeof(T) == 4) return KI <= 64 && NT == 1 ? 3 : KI <= 128 ? 2 : 1;
  return NT == 1 && KI <= (MODE == kLinOut ? 64 : 128) ? 3 : 2;
}
// Sum of the waves' values of row x.
template <int L>
__device__ __forceinline__ float lin_sum(const float (&red)[kLinWaves][L], int x) {
  return (red[0][x] + red[1][x]) + (red[2][x] + red[3][x]);
}

// What lies in LDS, in elements of 16 bits.  P takes the place of Q, which has
// been read by then.
template <typename T, int KI, int WO, int MODE>
struct LinTiles {
  static constexpr int L = LinTypes<T>::L, NP = LinTypes<T>::NP, NS = kLinPieces;
  static constexpr int kQ = 0, kP = 0;
  static constexpr int kQP = NP * L * KI > NS * L * L ? NP * L * KI : NS * L * L;
  static constexpr int kK = MODE == kLinState ? 0 : kQP;
  static constexpr int kV = kK + NP * L * KI;
  static constexpr int kEnd = kV + NP * L * WO;
};

// Which workgroup this is: `each` of them (roles, tiles) to a head and segment.
// Neighbouring ones lie on different XCDs, each with an L2 of its own: they
// are renumbered so that an XCD takes runs of them, the roles and tiles of up to
// eight heads of one key head, and what those read twice comes from its L2.
// (Longer runs leave XCDs idle where sequences differ in length: seven prompts
// in 6000 rows 274 us with one run an XCD, 176 without any.)
struct LinBlock {
  uint32_t each, sg, h, b;
};
__device__ __forceinline__ LinBlock lin_block(const LinArgs& a, uint32_t each) {
  const uint64_t all = (uint64_t)gridDim.x * gridDim.y * gridDim.z;
  uint32_t id = blockIdx.x + gridDim.x * (blockIdx.y + gridDim.y * blockIdx.z);
  if (all >= (uint64_t)1 << 32)
    return LinBlock{blockIdx.x % each, blockIdx.x / each, blockIdx.y, blockIdx.z};
  const uint32_t reps = a.Hv / a.Hk, run = each * (reps < 8 ? reps : 8);
  const uint32_t block = id / (8 * run) * (8 * run);
  if (block + 8 * run <= (uint32_t)all) {
    const uint32_t in = id - block;
    id = block + in % 8 * run + in / 8;
  }
  const uint32_t rest = id / each, h = rest % a.Hv, at = rest / a.Hv;
  return LinBlock{id - rest * each, at % a.segs, h, at / a.segs};
}

template <typename T, int KI, int NT, int MODE, bool VEC>
__device__ __forceinline__ void lin_chunk_run(const LinArgs& a, const LinRole& r, LinBlock at,
                                              uint16_t* lds) {
  constexpr int WO = 16 * NT * kLinWaves;
  using Z = LinTiles<T, KI, WO, MODE>;
  constexpr int L = Z::L, NP = Z::NP, NS = Z::NS, IT = L / 16, KS = KI / 32;
  constexpr bool OUT = MODE != kLinState, FLOW = MODE == kLinFlow;
  __shared__ __attribute__((aligned(16))) float2 Hs[L];  // in units of ln 2, hi + lo
  __shared__ __attribute__((aligned(16))) float cf[L], uf[L], pd[L];
  __shared__ float total_s, red[kLinWaves][L];
  __shared__ uint32_t part_s;  // rows of a pass (lin_part)
  __shared__ LinPass pass_s;
  __shared__ int odd_s[kLinWaves], odd_row[WO];
  const int wave = threadIdx.x >> 6;
  const int tile = at.each, sg = at.sg, h = at.h, b = at.b;
  const Span sp = span_of(a.spans, b, a.T, a.rows);
  const int begin = sg * a.seg;
  if ((sg > 0 || MODE == kLinState) && begin >= sp.len) return;
  const int len = sp.len - begin < a.seg ? sp.len - begin : a.seg;  // of this segment
  const int chunks = (len + L - 1) / L;
  const int64_t size = (int64_t)r.Ni * r.No, slot = lin_slot(a, sp, b, sg);
  const int o0 = tile * WO, wo = o0 + wave * 16 * NT;  // the wave's columns
  const int no = r.No - o0;

  uint16_t *Qt[NP], *Kt[NP], *Vt[NP], *Pt[NS];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    Qt[i] = lds + Z::kQ + i * L * KI;
    Kt[i] = lds + Z::kK + i * L * KI;
    Vt[i] = lds + Z::kV + i * L * WO;
  }
#pragma unroll
  for (int i = 0; i < NS; ++i) Pt[i] = lds + Z::kP + i * L * L;

  // The state: tile pair s (columns 32 s + 8 q + 4 k + v of Ni), columns lr.
  f4 S[2 * KS][NT];
  // (the lane is made opaque, so that no addresses stay in registers between
  // the loads and the stores: they would be as many as the state)
  auto each = [&](auto f) __attribute__((always_inline)) {
    int l = threadIdx.x & 63;
    asm volatile("" : "+v"(l));
    const int i0 = 8 * (l >> 4), o = wo + (l & 15);
    const int step_i = r.transposed ? r.No : 1, step_o = r.transposed ? 1 : r.Ni;
    const int at = i0 * step_i + o * step_o;
#pragma unroll
    for (int s = 0; s < 2 * KS; ++s)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int i = 32 * (s >> 1) + 4 * (s & 1) + v;
          S[s][nt][v] = f(S[s][nt][v], at + i * step_i + 16 * nt * step_o,
                          i0 + i < r.Ni && o + 16 * nt < r.No);
        }
  };
  const float* first = nullptr;
  if (r.first != nullptr)
    first = r.first + ((r.slots ? slot : (int64_t)b) * a.Hv + h) * size;
  each([&](float, int at, bool in) __attribute__((always_inline)) {
    return first != nullptr && in ? first[at] : 0.f;
  });
  auto put_state = [&](float* to) __attribute__((always_inline)) {
    each([&](float x, int at, bool in) __attribute__((always_inline)) {
      if (in) to[at] = x;
      return x;
    });
  };
  const bool save = r.save != nullptr && len > 0;
  if (save) put_state(r.save + (slot * a.Hv + h) * size);

  LinStage<T, KI> qs, ks;
  LinStage<T, WO> vs;
  float lg = 0.f;
  // Rows of the next tile, one tensor at a time, so that the requests do not
  // queue up: row x of a tile is step t0 + x, or t0 + L - 1 - x.
  const T* const Q = static_cast<const T*>(r.Q) + (int64_t)(h / r.dq) * r.Ni;
  const T* const K = static_cast<const T*>(r.K) + (int64_t)(h / r.dk) * r.Ni;
  const T* const V = static_cast<const T*>(r.V) + (int64_t)(h / r.dv) * r.No + o0;
  auto start = [&](int c) { return (r.reverse ? chunks - 1 - c : c) * L; };
  auto count = [&](int t0) { return len - t0 < L ? len - t0 : L; };
  auto fetch_q = [&](int c, int thread) __attribute__((always_inline)) {
    const int t0 = start(c), n = count(t0);
    const int64_t row = sp.first + begin + t0;
    if constexpr (OUT) qs.template load<VEC>(Q + row * r.sq, r.sq, n, r.Ni, thread);
    if (thread < L) {
      const int t = r.reverse ? L - 1 - thread : thread;
      lg = t < n ? lin_log_decay(a, row + t, h) : 0.f;
    }
  };
  auto fetch_k = [&](int c, int thread) __attribute__((always_inline)) {
    const int t0 = start(c);
    ks.template load<VEC>(K + (sp.first + begin + t0) * r.sk, r.sk, count(t0), r.Ni, thread);
  };
  auto fetch_v = [&](int c, int thread) __attribute__((always_inline)) {
    const int t0 = start(c);
    vs.template load<VEC>(V + (sp.first + begin + t0) * r.sv, r.sv, count(t0), no < WO ? no : WO,
                          thread);
  };
  if (chunks > 0) {
    fetch_q(0, threadIdx.x);
    fetch_k(0, threadIdx.x);
    fetch_v(0, threadIdx.x);
  }
  double all = 0.0;  // the segment's summed log decays (first wave)
  if (threadIdx.x == 0) pass_s = LinPass{0.f, 0, 0};

  for (int c = 0; c < chunks;) {
    // (opaque, so that addresses are formed where they are used and do not
    // fill the registers through the loop)
    int thread = threadIdx.x;
    asm volatile("" : "+v"(thread));
    const int lane = thread & 63, q = lane >> 4, lr = lane & 15;
    const int rows = lin_row_place<KI>(lane), prows = lin_row_place<L>(lane);
    const int kcols = lin_column_place<KI, true>(lane);
    const int vcols = lin_move<WO>(lin_column_place<WO, false>(lane), 16 * NT * wave);
    lds_barrier();  // the last tile has been read
    if constexpr (OUT) qs.store(Qt, r.reverse, thread);
    ks.store(Kt, r.reverse, thread);
    vs.store(Vt, r.reverse, thread);
    {
      const bool odd = __any(vs.odd());
      if ((threadIdx.x & 63) == 0) odd_s[wave] = odd;
    }
    if (threadIdx.x < 64) {
      double x = threadIdx.x < L ? (double)lg : 0.0;
      x = x < kLeastLog ? kLeastLog : x;  // (NaN stays)
      uint32_t part = lin_part(0, L, true);
      if (__builtin_expect(__any(x > 0.0), 0)) part = lin_pass<L>(x, pass_s, r.reverse);
      if (threadIdx.x == 0) part_s = part;
      const double sum = lin_prefix_sum(x);
      const double earlier = lin_dpp<0x138, 0xF>(sum);  // wave_shr:1
      const double end = __shfl(sum, 63, 64);
      if constexpr (!OUT) all += __any(x <= kLeastLog) ? end - __builtin_inf() : end;
      const bool before = threadIdx.x < (part & 255), in = !before && threadIdx.x < (part >> 8 & 255);
      if (threadIdx.x < L) {
        // (a difference to x would carry a NaN x into its own row)
        const double H = r.reverse ? earlier : sum;
        const double H2 = H * 1.4426950408889634;
        const float hi = (float)H2;
        // (rows before the pass reach nothing in it, those behind not the state)
        Hs[threadIdx.x] = before ? float2{1e30f, 0.f} : float2{hi, (float)(H2 - (double)hi)};
        cf[threadIdx.x] = r.cs * lin_exp(H);
        uf[threadIdx.x] = in ? r.us * lin_exp(end - H) : 0.f;
        if (threadIdx.x == 0) total_s = lin_exp(end);
      }
    }
    lds_barrier();
    const int t0 = start(c);
    const uint32_t part = __builtin_amdgcn_readfirstlane(part_s);
    const int x0 = part & 255, x1 = part >> 8 & 255;
    const int next = c + (int)(part >> 16);
    const bool more = next < chunks;
    // What is not finite in V may reach its own row and later ones only, but a
    // matrix product multiplies it with the zeros of P above the diagonal too.
    // It is taken out, and each column's outputs from its first such row on,
    // and the column's state, are made NaN instead.  (Looking for them cost 0 to
    // 4% of a pass in bf16, 8% of the small one in fp32, when it was added:
    // training of 2048 steps, heads 16/64 of 192/128, 473 us, 456 without.)
    const bool odd = __builtin_amdgcn_readfirstlane(odd_s[0] | odd_s[1] | odd_s[2] | odd_s[3]);
    if (__builtin_expect(odd, 0)) {
      if (threadIdx.x < WO) {
        int first = L;
#pragma clang loop unroll(disable)
        for (int x = L - 1; x >= 0; --x) {
          const int at = lin_at<WO>(x, threadIdx.x);
          if ((Vt[0][at] & 0x7fff) >= kLinInf) {
            first = x;
#pragma unroll
            for (int i = 0; i < NP; ++i) Vt[i][at] = 0;
          }
        }
        odd_row[threadIdx.x] = first;
      }
      lds_barrier();
    }
    if (more) fetch_q(next, thread);

    f4 acc[IT][NT];
    if constexpr (OUT) {
      // P: the tiles of 16 x 16 that its products below read (row it, columns
      // up to 16 (it | 1) + 15) dealt to the waves, their products first and
      // their decays behind S Q, which leaves the matrix cores time for them
      constexpr int PT = IT == 4 ? 12 : 4, PW = (PT + kLinWaves - 1) / kLinWaves;
      f4 p[PW];
      int pi[PW], pj[PW];
#pragma unroll
      for (int k = 0; k < PW; ++k) {
        // (past the last: that one again)
        const int t = PW * wave + k < PT ? PW * wave + k : PT - 1;
        pi[k] = IT == 4 ? (t >= 2) + (t >= 4) + (t >= 8) : t >> 1;
        pj[k] = t < 4 ? t & 1 : t & 3;
        p[k] = f4{0.f, 0.f, 0.f, 0.f};
      }
#pragma unroll
      for (int s = 0; s < KS; ++s) {
#pragma unroll
        for (int k = 0; k < PW; ++k) {
          uint4 ka[NP], qb[NP];
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            ka[i] = lin_rows<KI>(Kt[i], rows, 16 * pj[k], 32 * s);
            qb[i] = lin_rows<KI>(Qt[i], rows, 16 * pi[k], 32 * s);
          }
          p[k] = lin_mfma(ka, qb, p[k]);
        }
      }
      if (more) fetch_k(next, thread);
      // out <- S Q, scaled by cf
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int it = 0; it < IT; ++it)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) acc[it][nt] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        uint4 sa[NT][NS];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) lin_split(S[2 * s][nt], S[2 * s + 1][nt], sa[nt]);
#pragma unroll
        for (int it = 0; it < IT; ++it) {
          uint4 qb[NP];
#pragma unroll
          for (int i = 0; i < NP; ++i) qb[i] = lin_rows<KI>(Qt[i], rows, 16 * it, 32 * s);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) acc[it][nt] = lin_mfma(sa[nt], qb, acc[it][nt]);
        }
      }
      __builtin_amdgcn_s_setprio(0);
      lds_barrier();  // Q has been read
      const int pput = lin_at<L>(lr, 4 * q);
#pragma unroll
      for (int k = 0; k < PW; ++k) {
        const int i = 16 * pi[k] + lr, j = 16 * pj[k] + 4 * q;
        const float2 Hi = Hs[i];
        const float4 H01 = *reinterpret_cast<const float4*>(Hs + j);
        const float4 H23 = *reinterpret_cast<const float4*>(Hs + j + 2);
        const float hi[4] = {H01.x, H01.z, H23.x, H23.z}, lo[4] = {H01.y, H01.w, H23.y, H23.w};
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const float x = r.ps * p[k][v];
          if (FLOW && i == j + v) pd[i] = x;
          // (a mask, as a choice becomes a branch around the exponential)
          const int below = i - (FLOW ? 1 : 0) - (j + v);
          p[k][v] = __uint_as_float(
              __float_as_uint(x * exp2_hw((Hi.x - hi[v]) + (Hi.y - lo[v]))) & ~(below >> 31));
        }
        uint4 pieces[NS];
        lin_split(p[k], f4{0.f, 0.f, 0.f, 0.f}, pieces);
#pragma unroll
        for (int n = 0; n < NS; ++n)
          *reinterpret_cast<uint2*>(Pt[n] + 16 * L * pi[k] + lin_move<L>(pput, 16 * pj[k])) =
              uint2{pieces[n].x, pieces[n].y};
      }
#pragma unroll
      for (int it = 0; it < IT; ++it) {
        const float x = cf[16 * it + lr];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) acc[it][nt] *= x;
      }
      lds_barrier();  // P is whole
    } else {
      if (more) fetch_k(next, thread);
    }
    if (more) fetch_v(next, thread);
    // the rows that the flows multiply with, in time for the end of the tile
    const int n = count(t0), lane_row = r.reverse ? 15 - lr : lr, o = wo + 4 * q;
    const int64_t row = sp.first + begin + t0;
    LinQuad<VEC, T> with[FLOW ? IT : 1][FLOW ? NT : 1];
    if constexpr (FLOW) {
      const Buffer R = buffer_of(r.R, (row * r.sr + (int64_t)(h / r.dr) * r.No) * sizeof(T),
                                 ((int64_t)(n - 1) * r.sr + r.No) * sizeof(T));
#pragma unroll
      for (int it = 0; it < IT; ++it)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int t = r.reverse ? L - 16 - 16 * it : 16 * it;
          with[it][nt].load(R, (uint32_t)(lane_row * (uint32_t)r.sr + o) * sizeof(T),
                            (uint32_t)(t * (uint32_t)r.sr + 16 * nt) * sizeof(T),
                            r.No - o - 16 * nt);
        }
    }
    {
      const float x = total_s;
#pragma unroll
      for (int s = 0; s < 2 * KS; ++s)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) S[s][nt] *= x;
    }
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int k = 0; k < L / 32; ++k) {
      uint4 vo[NT][NP], vu[NT][NS];
      const f4 u0 = *reinterpret_cast<const f4*>(uf + 32 * k + 8 * q);
      const f4 u1 = *reinterpret_cast<const f4*>(uf + 32 * k + 8 * q + 4);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        f4 x, y;
#pragma unroll
        for (int i = NP - 1; i >= 0; --i) {
          const uint4 w = vo[nt][i] = lin_columns<WO>(Vt[i], vcols, 32 * k, 16 * nt);
          const f4 wx = lin_unpack(uint2{w.x, w.y}), wy = lin_unpack(uint2{w.z, w.w});
          x = i == NP - 1 ? wx : x + wx;
          y = i == NP - 1 ? wy : y + wy;
        }
        lin_split(x * u0, y * u1, vu[nt]);
      }
      if constexpr (OUT) {
#pragma unroll
        for (int it = 2 * k; it < IT; ++it) {
          uint4 pb[NS];
#pragma unroll
          for (int n = 0; n < NS; ++n) pb[n] = lin_rows<L>(Pt[n], prows, 16 * it, 32 * k);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) acc[it][nt] = lin_mfma(vo[nt], pb, acc[it][nt]);
        }
      }
#pragma unroll
      for (int s = 0; s < 2 * KS; ++s) {
        uint4 ka[NP];
#pragma unroll
        for (int i = 0; i < NP; ++i)
          ka[i] = lin_columns<KI>(Kt[i], kcols, 32 * k, 32 * (s >> 1) + 4 * (s & 1));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) S[s][nt] = lin_mfma(ka, vu[nt], S[s][nt]);
      }
    }
    __builtin_amdgcn_s_setprio(0);
    if (__builtin_expect(odd, 0)) {
      const float nan = __builtin_nanf("");
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int col = 16 * NT * wave + 16 * nt;
        if (odd_row[col + lr] < x1)
#pragma unroll
          for (int s = 0; s < 2 * KS; ++s) S[s][nt] = f4{nan, nan, nan, nan};
        if constexpr (OUT) {
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const int first = odd_row[col + 4 * q + v];
#pragma unroll
            for (int it = 0; it < IT; ++it)
              if (16 * it + lr >= first) acc[it][nt][v] = nan;
          }
        }
      }
    }
    if constexpr (OUT) {
      const int wide = a.Hv * r.No;
      // rows past the sequence's end are past the buffers'
      const int es = r.out != nullptr ? (int)sizeof(T) : 4;
      const Buffer out = buffer_of(r.out != nullptr ? r.out : r.part,
                                   (row * wide + (int64_t)h * r.No) * es,
                                   ((int64_t)(n - 1) * wide + r.No) * es);
      const int vput = lin_move<WO>(lin_at<WO>(lr, 4 * q), 16 * NT * wave);
#pragma unroll
      for (int it = 0; it < IT; ++it) {
        const int x = 16 * it + lr;
        float flow = 0.f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if constexpr (FLOW) {
            const f4 w = with[it][nt].get();
#pragma unroll
            for (int v = 0; v < 4; ++v) flow = fmaf(w[v], acc[it][nt][v], flow);
            // the step's own term
            f4 own;
#pragma unroll
            for (int i = NP - 1; i >= 0; --i) {
              const f4 y = lin_unpack(*reinterpret_cast<const uint2*>(
                  Vt[i] + 16 * WO * it + lin_move<WO>(vput, 16 * nt)));
              own = i == NP - 1 ? y : own + y;
            }
            acc[it][nt] += own * pd[x];
          }
        }
        if constexpr (FLOW) {
          flow = swap16_sum(flow, flow);
          flow = swap32_sum(flow, flow);
          if (q == 0) red[wave][x] = flow;
        }
      }
      auto put = [&](auto type) __attribute__((always_inline)) {
        using O = decltype(type);
#pragma unroll
        for (int it = 0; it < IT; ++it)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const int t = r.reverse ? L - 16 - 16 * it : 16 * it, x = 16 * it + lr;
            lin_put<VEC, O>(out, (uint32_t)(lane_row * wide + o) * sizeof(O),
                            (uint32_t)(t * wide + 16 * nt) * sizeof(O), acc[it][nt],
                            x >= x0 && x < x1 ? r.No - o - 16 * nt : 0);
          }
      };
      if (r.out != nullptr)
        put(T{});
      else
        put(float{});
      if constexpr (FLOW) {
        lds_barrier();
        const int x = thread, t = r.reverse ? L - 1 - x : x;
        if (x >= x0 && x < x1 && t < n)
          r.flow[((int64_t)tile * a.Hv + h) * a.rows + row + t] = lin_sum<L>(red, x);
      }
    }
    c = next;
  }
  if constexpr (MODE == kLinState) {
    put_state(r.local + ((slot + (r.reverse ? 0 : 1)) * a.Hv + h) * size);
    if (threadIdx.x == 0 && tile == 0) r.decay[slot * a.Hv + h] = all;
  }
  if (r.last != nullptr) put_state(r.last + ((int64_t)b * a.Hv + h) * size);
  if (save) put_state(r.save + ((slot + 1) * a.Hv + h) * size);
}

template <typename T, int KI, int NT, int MODE, bool VEC>
__global__ __launch_bounds__(64 * kLinWaves, (lin_waves<T>(KI, NT, MODE))) void lin_chunk_kernel(
    LinArgs a, LinRole r) {
  __shared__ __attribute__((aligned(16))) uint16_t
      lds[LinTiles<T, KI, 16 * NT * kLinWaves, MODE>::kEnd];
  lin_chunk_run<T, KI, NT, MODE, VEC>(a, r, lin_block(a, r.tiles), lds);
}

// dq, dk and dv in one launch, where their widths take the same instance.
struct LinRoles {
  LinRole r[3];
};
template <typename T, int KI, int NT, int MODE, bool VEC>
__global__ __launch_bounds__(64 * kLinWaves, (lin_waves<T>(KI, NT, MODE))) void lin_chunks_kernel(
    LinArgs a, LinRoles roles) {
  __shared__ __attribute__((aligned(16))) uint16_t
      lds[LinTiles<T, KI, 16 * NT * kLinWaves, MODE>::kEnd];
  LinBlock at = lin_block(a, 3 * roles.r[0].tiles);
  const uint32_t role = at.each % 3;
  at.each /= 3;
  if (MODE == kLinFlow && role == 2)
    lin_chunk_run<T, KI, NT, kLinOut, VEC>(a, roles.r[2], at, lds);
  else
    lin_chunk_run<T, KI, NT, MODE, VEC>(a, roles.r[role], at, lds);
}

// The instances: widths of 64 to 256 contracted, 64 or 128 columns of output.
template <typename T, bool VEC>
hipError_t lin_chunk(const LinArgs& a, const LinRole& r, int mode, hipStream_t s);
// dq, dk and dv (whose mode is kLinOut) of one call.
template <typename T, bool VEC>
hipError_t lin_chunks(const LinArgs& a, const LinRoles& r, int mode, hipStream_t s);

}  // namespace gdr
