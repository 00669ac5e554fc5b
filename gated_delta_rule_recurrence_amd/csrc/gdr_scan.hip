// Selective state space scan on gfx950.  Per sequence, channel c (in group g
// of G) and state n, with fp32 states:
//   delta = softplus(dt + dt_bias),  a = exp(delta A[c][n]),
//   h_t = a h_{t-1} + delta u B_t[g][n],
//   y_t = (sum_n C_t[g][n] h_t + D u) silu(z).
// Adjoint, with o = dy silu(z) and the carried E_t = dL/dh_t:
//   E_t = o C_t + a_{t+1} E_{t+1},  dC_t = sum_c o h_t,
//   dB_t = sum_c E_t delta u,  du = D o + delta sum_n E_t B_t,
//   ddelta = sum_n E_t (u B_t + A a h_{t-1}),  dA = sum_t E_t delta a h_{t-1},
//   ddt = ddelta sigmoid(dt + dt_bias),  dS0 = a_1 E_1.
// Every state and step takes one exponential (two of a vector unit's turns)
// and 4 (forward) or 12 (backward) products and sums: bound by the vector
// units, not by HBM.  Measured (bf16, N = 16, at 39 T lane-operations/s): 4 x
// 4096 x 4096, forward unsplit 427 us, 16 operations' time a state and step
// (57% busy, one wave a SIMD), backward 191 + 754 us, 7 and 28 (93 and 99%
// busy).  Of the backward's 28 the formula takes 14, the sums of dB and dC
// over channels 4, preparing the steps 4, sums over states and broadcasts 3.
//
// Mapping: the four lanes of a DPP quad share a channel, NPL states each; a
// wave has 16 channels, a workgroup 64.  Time runs in tiles of TT steps: lane
// r of a quad loads and prepares (softplus, gate) steps 4 q + r of its
// channel, the recurrence then broadcasts them inside the quad, and sums over
// n go back to the step's lane in two exchanges.  B and C come from LDS,
// where four addresses serve the wave.
//
// Long sequences with few channels are split into chunks of L steps that run
// side by side: a first pass leaves every chunk's end state from a zero
// start (edge) and its sum of delta (dsum); the main pass joins those of the
// chunks before its own, h_in(j + 1) = exp(A dsum_j) h_in(j) + edge_j, and
// starts from there.  The backward joins the adjoint the same way.
#include "gdr_layer.h"

namespace gdr {
namespace {

// Registers for n waves a SIMD and no fewer: for the eight that fit, the
// compiler orders the recurrence's loads and exponentials so tightly that the
// adjoint pass takes 227 us instead of 201 (4 x 4096 x 4096; at four, as at
// six).  Packed prompts (five in 4100 rows of 4096): 149 us at four, 159 at
// six, 152 at five or three.
#define SCAN_WAVES(n) __attribute__((amdgpu_waves_per_eu(n, n)))

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kChannels = 64;  // of one workgroup
constexpr int kMaxChunks = 64;
constexpr int kMaxStep = 4;    // steps that scan_step_kernel takes

template <int NPL>
constexpr int tile_steps() {
  return NPL <= 4 ? 16 : 64 / NPL;
}

// Steps between saved states: what the backward keeps in registers at a time
// (the states and decays of that many steps).
template <int NPL>
constexpr int save_steps() {
  return NPL <= 4 ? 8 : 4;
}

template <int K>
__device__ __forceinline__ float quad_bcast(float x) {
  return dpp<K * 0x55>(x);
}
// Lane r of a quad receives the sum over the quad's lanes of argument r.
__device__ __forceinline__ float quad_scatter_sum(const float (&a)[4], int r) {
  const bool b0 = r & 1, b1 = r & 2;
  float k0 = b0 ? a[1] : a[0], k1 = b0 ? a[3] : a[2];
  k0 += dpp<kDppQuadSwap1>(b0 ? a[0] : a[1]);
  k1 += dpp<kDppQuadSwap1>(b0 ? a[2] : a[3]);
  float k = b1 ? k1 : k0;
  k += dpp<kDppQuadSwap2>(b1 ? k0 : k1);
  return k;
}
__device__ __forceinline__ float quad_sum(float x) {
  x += dpp<kDppQuadSwap1>(x);
  x += dpp<kDppQuadSwap2>(x);
  return x;
}

// Sum of a[i] over the 16 quads of a wave (lanes of equal r).  CNT values go
// in; values CNT / 4 * (l / 16) .. of lane l come out (CNT = 2: value l / 32).
template <int CNT>
__device__ __forceinline__ void quads_scatter_sum(const float (&a)[CNT],
                                                  float (&o)[CNT > 2 ? CNT / 4 : 1]) {
  float h[CNT / 2];
#pragma unroll
  for (int i = 0; i < CNT / 2; ++i) h[i] = swap32_sum(a[i], a[i + CNT / 2]);
#pragma unroll
  for (int i = 0; i < (CNT > 2 ? CNT / 4 : 1); ++i) {
    float x = swap16_sum(h[i], CNT > 2 ? h[i + CNT / 4] : h[i]);
    x += dpp<0x124>(x);  // row_ror:4
    x += dpp<0x128>(x);  // row_ror:8
    o[i] = x;
  }
}

// Where a thread stands: its channel, and its chunk of its sequence.
struct Place {
  Span sp;
  int b, g, tile_in_group, c, r, wave;
  bool cok;
  int begin, end;  // steps of the chunk
  int j, last;     // chunk, last chunk that has steps (0 for an empty sequence)
};
// (The divisions cost a short call more than its loads: skipped where there
// is one chunk, one group.)
__device__ __forceinline__ Place place_of(const ScanArgs& a, int ctiles) {
  Place p;
  p.b = blockIdx.y;
  p.sp = span_of(a.spans, p.b, a.T, a.rows);
  // the same for the whole workgroup: kept in scalar registers
  p.sp.first = __builtin_amdgcn_readfirstlane((int)p.sp.first);
  p.sp.len = __builtin_amdgcn_readfirstlane(p.sp.len);
  int ct = blockIdx.x;
  p.j = p.last = 0;
  if (a.chunks > 1) {
    p.j = ct / ctiles;
    ct -= p.j * ctiles;
    p.last = p.sp.len > 0 ? (p.sp.len - 1) / a.chunk : 0;
  }
  int Cg = a.C;
  p.g = 0;
  p.tile_in_group = ct;
  if (a.G > 1) {
    const int tpg = ctiles / a.G;
    p.g = ct / tpg;
    p.tile_in_group = ct - p.g * tpg;
    Cg = a.C / a.G;
  }
  p.wave = threadIdx.x >> 6;
  p.r = threadIdx.x & 3;
  const int in = p.tile_in_group * kChannels + (threadIdx.x >> 2);
  p.cok = in < Cg;
  p.c = p.g * Cg + (p.cok ? in : 0);
  const int64_t b0 = (int64_t)p.j * a.chunk, b1 = b0 + a.chunk;
  p.begin = (int)(b0 < p.sp.len ? b0 : p.sp.len);
  p.end = (int)(b1 < p.sp.len ? b1 : p.sp.len);
  return p;
}
// Slots of a sequence's chunks (tiles) of n steps: distinct for ascending
// disjoint spans, below rows / n + B + 1 for any.
__device__ __forceinline__ int64_t slot_of(const Span& sp, int b, int n, int j) {
  return sp.first / n + b + j;
}

// Rows and states go through buffer resources: a base that the whole
// workgroup shares, 32 bits of offset per lane, and a bound past which loads
// give zero and stores are dropped.  That is what steps past a sequence's end
// and lanes without a channel (kNoLane) need, with no masks.  The base is the
// chunk's first row, so the offsets of its rows, and of its saved states,
// have to stay below 2^31 bytes (scan_chunk sees to that): kNoLane plus any
// of them is then past every bound and does not wrap.
constexpr uint32_t kNoLane = 0x80000000u;
template <typename T>
__device__ __forceinline__ T get(Buffer b, uint32_t offset);
template <>
__device__ __forceinline__ bf16 get<bf16>(Buffer b, uint32_t offset) {
  return bf16{(uint16_t)__builtin_amdgcn_raw_buffer_load_b16(b.resource(), (int)offset, 0, 0)};
}
template <>
__device__ __forceinline__ float get<float>(Buffer b, uint32_t offset) {
  return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(b.resource(), (int)offset, 0, 0));
}
template <typename T>
__device__ __forceinline__ void put(Buffer b, uint32_t offset, float x);
template <>
__device__ __forceinline__ void put<bf16>(Buffer b, uint32_t offset, float x) {
  __builtin_amdgcn_raw_buffer_store_b16((unsigned short)cvt_pk_bf16(x, x), b.resource(),
                                        (int)offset, 0, 0);
}
template <>
__device__ __forceinline__ void put<float>(Buffer b, uint32_t offset, float x) {
  __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x), b.resource(), (int)offset, 0, 0);
}

// A lane's NPL states of its channel, in the user's [C][N] layout
template <int NPL>
__device__ __forceinline__ void load_states(const float* p, int N, int r, bool ok,
                                            float (&h)[NPL]) {
  if (NPL % 4 == 0 && N == 4 * NPL) {  // whole vectors
#pragma unroll
    for (int k = 0; k < NPL; k += 4) {
      const f4 v = ok ? *reinterpret_cast<const f4*>(p + r * NPL + k) : f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int e = 0; e < 4; ++e) h[k + e < NPL ? k + e : 0] = v[e];
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < NPL; ++i) h[i] = ok && r * NPL + i < N ? p[r * NPL + i] : 0.f;
}
template <int NPL>
__device__ __forceinline__ void store_states(float* p, int N, int r, bool ok,
                                             const float (&h)[NPL]) {
  if (NPL % 4 == 0 && N == 4 * NPL) {
    if (!ok) return;
#pragma unroll
    for (int k = 0; k < NPL; k += 4) {
      f4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = h[k + e < NPL ? k + e : 0];
      *reinterpret_cast<f4*>(p + r * NPL + k) = v;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < NPL; ++i)
    if (ok && r * NPL + i < N) p[r * NPL + i] = h[i];
}
// and in a padded slot [C][4 NPL] of a library buffer
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
template <int NPL>
__device__ __forceinline__ Buffer slot_buffer(const float* p, int64_t slot, int C) {
  const int64_t bytes = (int64_t)C * 16 * NPL;  // C <= 2^20: at most 2^28
  return buffer_of(p, slot * bytes, bytes);
}
template <int NPL>
__device__ __forceinline__ void get_states(Buffer b, uint32_t o, float (&h)[NPL]) {
  if constexpr (NPL == 1) {
    h[0] = get<float>(b, o);
  } else if constexpr (NPL == 2) {
    const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(b.resource(), (int)o, 0, 0);
    h[0] = __uint_as_float(v[0]);
    h[1] = __uint_as_float(v[1]);
  } else {
#pragma unroll
    for (int k = 0; k < NPL; k += 4) {
      const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(b.resource(), (int)(o + 4 * k), 0, 0);
#pragma unroll
      for (int e = 0; e < 4; ++e) h[k + e] = __uint_as_float(v[e]);
    }
  }
}
template <int NPL>
__device__ __forceinline__ void put_states(Buffer b, uint32_t o, const float (&h)[NPL]) {
  if constexpr (NPL == 1) {
    put<float>(b, o, h[0]);
  } else if constexpr (NPL == 2) {
    __builtin_amdgcn_raw_buffer_store_b64(u32x2{__float_as_uint(h[0]), __float_as_uint(h[1])},
                                          b.resource(), (int)o, 0, 0);
  } else {
#pragma unroll
    for (int k = 0; k < NPL; k += 4)
      __builtin_amdgcn_raw_buffer_store_b128(
          u32x4{__float_as_uint(h[k]), __float_as_uint(h[k + 1]), __float_as_uint(h[k + 2]),
                __float_as_uint(h[k + 3])},
          b.resource(), (int)(o + 4 * k), 0, 0);
  }
}

// The loads of a tile: this lane's steps of its channel, and this thread's
// element of B and C; zeros past the sequence's end.  The offsets walk from
// tile to tile.
template <typename T, int NPL, int TT, bool IN, bool OUT, bool DY>
struct Tile {
  static constexpr int Q = TT / 4, NP = 4 * NPL;
  struct Raw {
    T u[Q], dt[Q], z[Q], dy[Q];
    T bm, cm;
  };
  Buffer bu, bdt, bz, bdy, bb, bc;   // the chunk's rows
  uint32_t su, sdt, sz, sd, sb, sc;  // bytes from row to row
  uint32_t ou, odt, oz, od, ob, oc;  // this lane in the first four rows of the tile at hand

  // At the tile that starts t0 steps into the chunk.
  __device__ __forceinline__ void init(const ScanArgs& a, const Place& p, int t0) {
    const int64_t row = p.sp.first + p.begin;
    auto rows = [&](const void* q, int64_t stride, uint32_t& step) {
      step = (uint32_t)stride * (uint32_t)sizeof(T);
      return buffer_of(q, row * (int64_t)step,
                       q != nullptr ? (int64_t)(p.end - p.begin) * step : 0);
    };
    bu = rows(a.u, a.u_stride, su);
    bdt = rows(a.dt, a.dt_stride, sdt);
    bz = rows(a.z, a.z_stride, sz);
    bdy = rows(a.dy, a.C, sd);
    bb = rows(a.Bm, a.b_stride, sb);
    bc = rows(a.Cm, a.c_stride, sc);
    auto lane = [&](uint32_t step) {
      return t0 * step + (p.cok ? p.r * step + p.c * (uint32_t)sizeof(T) : kNoLane);
    };
    ou = lane(su);
    odt = lane(sdt);
    oz = lane(sz);
    od = lane(sd);
    const uint32_t t = threadIdx.x / NP, n = threadIdx.x % NP;
    const bool ok = t < TT && (int)n < a.N;
    const uint32_t on = (p.g * a.N + n) * (uint32_t)sizeof(T);
    ob = t0 * sb + (ok ? t * sb + on : kNoLane);
    oc = t0 * sc + (ok ? t * sc + on : kNoLane);
  }
  __device__ __forceinline__ void load(Raw& w) const {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      if (IN) w.u[q] = get<T>(bu, ou + 4 * q * su);
      w.dt[q] = get<T>(bdt, odt + 4 * q * sdt);
      if (OUT) w.z[q] = get<T>(bz, oz + 4 * q * sz);
      if (DY) w.dy[q] = get<T>(bdy, od + 4 * q * sd);
    }
    if (IN) w.bm = get<T>(bb, ob);
    if (OUT) w.cm = get<T>(bc, oc);
  }
  // Moves the loads one tile on or back.
  template <int WAY>
  __device__ __forceinline__ void advance() {
    if (IN) ou += WAY * TT * su;
    odt += WAY * TT * sdt;
    if (OUT) oz += WAY * TT * sz;
    if (DY) od += WAY * TT * sd;
    if (IN) ob += WAY * TT * sb;
    if (OUT) oc += WAY * TT * sc;
  }
  static __device__ __forceinline__ void stage(const Raw& w, float* bs, float* cs) {
    if (TT * NP < kThreads && threadIdx.x >= TT * NP) return;
    if (IN) bs[threadIdx.x] = to_f32(w.bm);
    if (OUT) cs[threadIdx.x] = to_f32(w.cm);
  }
};

// delta of a raw step; 0, an identity step, outside the sequence.
__device__ __forceinline__ float delta_of(float raw, int plus, bool ok) {
  const float sp = softplus(raw);  // (not under the condition: a branch per step)
  const float d = plus ? sp : raw;
  return ok ? d : 0.f;
}

template <int NPL>
__device__ __forceinline__ void load_rates(const ScanArgs& a, const Place& p, float (&A)[NPL]) {
  load_states<NPL>(a.A + (int64_t)p.c * a.N, a.N, p.r, p.cok, A);
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    A[i] *= kLog2e;
    // an infinite rate becomes the largest one: a step past the sequence's
    // end has delta = 0, and its decay has to be 1
    A[i] = __builtin_isinf(A[i]) ? __builtin_copysignf(3.402823466e38f, A[i]) : A[i];
  }
}

// A sequence of several chunks keeps a copy of the state it starts from (the
// backward: of the adjoint it starts from) in the slot that no chunk's end
// uses, the last (the first), written by the first pass: the main pass then
// reads neither S0 nor dS_T while other workgroups of it write S_T or dS0,
// which may be the same memory.
template <int NPL>
__device__ __forceinline__ void start_states(const ScanArgs& a, const Place& p, const float* given,
                                             int slot, uint32_t oh, float (&h)[NPL]) {
  if (p.last > 0 && given != nullptr)
    get_states<NPL>(slot_buffer<NPL>(a.edge, slot_of(p.sp, p.b, a.chunk, slot), a.C), oh, h);
  else
    load_states<NPL>(given + ((int64_t)p.b * a.C + p.c) * a.N, a.N, p.r,
                     p.cok && given != nullptr, h);
}
template <int NPL>
__device__ __forceinline__ void copy_start(const ScanArgs& a, const Place& p, const float* given,
                                           int slot, uint32_t oh) {
  if (given == nullptr) return;
  float h[NPL];
  load_states<NPL>(given + ((int64_t)p.b * a.C + p.c) * a.N, a.N, p.r, p.cok, h);
  put_states<NPL>(slot_buffer<NPL>(a.edge, slot_of(p.sp, p.b, a.chunk, slot), a.C), oh, h);
}

// The state before chunk j (FWD), or the adjoint behind it: the chunks' local
// ones joined in the order of the recurrence, h <- exp(A dsum) h + edge, eight
// chunks' loads in flight (four with more than 4 states a lane).  Every
// workgroup joins for itself: kMaxChunks keeps that shorter than a kernel
// between the passes would take (5 to 8 us).
template <bool FWD, int NPL>
__device__ __forceinline__ void join_chunks(const ScanArgs& a, const Place& p, uint32_t oh,
                                            const float (&A)[NPL], float (&h)[NPL]) {
  const int64_t slot_bytes = (int64_t)a.C * NPL * 16;
  const int64_t s0 = slot_of(p.sp, p.b, a.chunk, 0);
  const char* const edge = reinterpret_cast<const char*>(a.edge) + s0 * slot_bytes;
  const float* const dsum = a.dsum + s0 * a.C + p.c;
  const int n = FWD ? p.j : p.last - p.j;
  constexpr int U = NPL <= 4 ? 8 : 4;
  for (int k0 = 0; k0 < n; k0 += U) {
    // (all loads first, with none under a condition, which would put a wait
    // between them; a chunk past the last counts as no steps)
    float e[U][NPL], d[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int at = k0 + k < n ? k0 + k : n - 1;
      const int64_t i = FWD ? at : p.last - at;
      get_states<NPL>(buffer_of(edge, i * slot_bytes, slot_bytes), oh, e[k]);
      d[k] = dsum[i * a.C];
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const bool in = k0 + k < n;
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        const float next = fmaf(exp2_hw(A[i] * d[k]), h[i], e[k][i]);
        h[i] = in ? next : h[i];
      }
    }
  }
}

// EDGE: the first pass (end state of every chunk but the last from a zero
// start); else the pass that writes y.
template <typename T, int NPL, bool EDGE>
__global__ __launch_bounds__(kThreads)
SCAN_WAVES((NPL <= 8 ? 4 : 3)) void scan_fwd_kernel(ScanArgs a, int ctiles) {
  constexpr int TT = tile_steps<NPL>(), HT = save_steps<NPL>();
  using L = Tile<T, NPL, TT, true, !EDGE, false>;
  constexpr int Q = L::Q, NP = L::NP;
  __shared__ __align__(16) float Bs[2][TT * NP], Cs[2][EDGE ? 4 : TT * NP];
  const Place p = place_of(a, ctiles);
  if (p.j > p.last) return;
  const int r = p.r;
  // this lane's states in a slot
  const uint32_t oh = p.cok ? (uint32_t)(p.c * NP + r * NPL) * 4u : kNoLane;
  if (EDGE && p.j == p.last) {
    if (p.last > 0) copy_start<NPL>(a, p, a.S0, p.last, oh);
    return;
  }
  float A[NPL], h[NPL];
  load_rates<NPL>(a, p, A);
  const float bias = a.dt_bias != nullptr ? a.dt_bias[p.c] : 0.f;
  const float D = a.D != nullptr ? a.D[p.c] : 0.f;
  if (EDGE) {
#pragma unroll
    for (int i = 0; i < NPL; ++i) h[i] = 0.f;
  } else {
    start_states<NPL>(a, p, a.S0, p.last, oh, h);
    join_chunks<true, NPL>(a, p, oh, A, h);
  }
  float sum = 0.f;
  // Loads of two tiles in flight: at one wave a SIMD a tile's arithmetic is
  // shorter than the way to memory (4 x 4096 x 4096, unsplit: 444 us, 456 with
  // one; 4 x 2048 x 4096 with 4 states: 196, 228).  The first passes have the
  // waves to hide it and lose 5 to 10% to the second set of registers.
  constexpr int kAhead = EDGE ? 1 : 2;
  L in;
  in.init(a, p, 0);
  uint32_t oy = in.od;
  typename L::Raw raw[kAhead];
  const int steps = p.end - p.begin;
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    if (k * TT < steps) in.load(raw[k]);
    in.template advance<1>();
  }
  const Buffer by = buffer_of(a.y, (p.sp.first + p.begin) * (int64_t)in.sd, (int64_t)steps * in.sd);
  // the saved states from this chunk's first on, of which this lane's next
  const int64_t slot_bytes = (int64_t)a.C * NP * 4;
  const Buffer saved =
      buffer_of(a.ckpt, slot_of(p.sp, p.b, HT, p.begin / HT) * slot_bytes,
                !EDGE && a.ckpt != nullptr ? (int64_t)((steps + HT - 1) / HT) * slot_bytes : 0);
  uint32_t osaved = oh;
  auto tile = [&](typename L::Raw& w, int t0, int buf) __attribute__((always_inline)) {
    // this lane's steps: delta, delta u, D u and the gate
    float dl[Q], du[Q], skip[Q], gate[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const float u = to_f32(w.u[q]);
      dl[q] = delta_of(to_f32(w.dt[q]) + bias, a.softplus, t0 + 4 * q + r < p.end);
      du[q] = dl[q] * u;
      if (EDGE) {
        sum += dl[q];
      } else {
        const float g = silu(to_f32(w.z[q]));
        skip[q] = D * u;
        gate[q] = a.z != nullptr ? g : 1.f;
      }
    }
    L::stage(w, Bs[buf], Cs[buf]);
    if (t0 + kAhead * TT < p.end) in.load(w);
    in.template advance<1>();
    __syncthreads();
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      if (!EDGE && 4 * q % HT == 0) {
        if (a.ckpt != nullptr) put_states<NPL>(saved, osaved, h);
        osaved += (uint32_t)slot_bytes;
      }
      float acc[4];
      auto step = [&](auto kk) __attribute__((always_inline)) {
        constexpr int k = decltype(kk)::value;
        const float dk = quad_bcast<k>(dl[q]), duk = quad_bcast<k>(du[q]);
        const float* const bp = Bs[buf] + (4 * q + k) * NP + r * NPL;
        const float* const cp = Cs[buf] + (EDGE ? 0 : (4 * q + k) * NP + r * NPL);
        acc[k] = 0.f;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
          h[i] = fmaf(exp2_hw(dk * A[i]), h[i], duk * bp[i]);
          if (!EDGE) acc[k] = fmaf(cp[i], h[i], acc[k]);
        }
      };
      step(std::integral_constant<int, 0>{});
      step(std::integral_constant<int, 1>{});
      step(std::integral_constant<int, 2>{});
      step(std::integral_constant<int, 3>{});
      if (!EDGE) {
        const float y = (skip[q] + quad_scatter_sum(acc, r)) * gate[q];
        put<T>(by, oy + 4 * q * in.sd, y);
      }
    }
    oy += TT * in.sd;
  };
  int buf = 0;
  for (int t0 = p.begin; t0 < p.end; t0 += kAhead * TT, buf ^= 1) {
    tile(raw[0], t0, kAhead > 1 ? 0 : buf);
    if (kAhead > 1 && t0 + TT < p.end) tile(raw[kAhead - 1], t0 + TT, 1);
  }
  if (EDGE) {
    put_states<NPL>(slot_buffer<NPL>(a.edge, slot_of(p.sp, p.b, a.chunk, p.j), a.C), oh, h);
    sum = quad_sum(sum);
    if (r == 0 && p.cok) a.dsum[slot_of(p.sp, p.b, a.chunk, p.j) * a.C + p.c] = sum;
  } else if (p.j == p.last && a.S_T != nullptr) {
    store_states<NPL>(a.S_T + ((int64_t)p.b * a.C + p.c) * a.N, a.N, r, p.cok, h);
  }
}

// A lane's NPL elements of a dense row of N (A, S0, B or C) as floats, zeros
// past N.  WHOLE: N = 4 NPL and the row starts on a multiple of four
// elements, so they are whole vectors.
template <typename T, int NPL, bool WHOLE>
__device__ __forceinline__ void get_row(Buffer b, uint32_t o, int r, int N, float (&x)[NPL]) {
  constexpr int kBytes = NPL * sizeof(T);
  const uint32_t at = o + r * kBytes;
  if constexpr (!WHOLE || kBytes < 4) {
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      x[i] = to_f32(get<T>(b, r * NPL + i < N ? at + i * (uint32_t)sizeof(T) : kNoLane));
  } else if constexpr (sizeof(T) == 4) {
    get_states<NPL>(b, at, x);
  } else {
    uint32_t w[NPL / 2];
    if constexpr (kBytes == 4) {
      w[0] = __builtin_amdgcn_raw_buffer_load_b32(b.resource(), (int)at, 0, 0);
    } else if constexpr (kBytes == 8) {
      const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(b.resource(), (int)at, 0, 0);
      w[0] = v[0];
      w[1] = v[1];
    } else {
#pragma unroll
      for (int k = 0; k < NPL / 2; k += 4) {
        const u32x4 v =
            __builtin_amdgcn_raw_buffer_load_b128(b.resource(), (int)(at + 4 * k), 0, 0);
#pragma unroll
        for (int e = 0; e < 4; ++e) w[k + e] = v[e];
      }
    }
#pragma unroll
    for (int i = 0; i < NPL / 2; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

// Sequences of at most kMaxStep steps (single tokens): the states stream once
// in and once out, so HBM bytes bound it.  The same quads, but no tiles, LDS
// or barriers: every lane prepares its channel's step and reads its states'
// B and C by itself.  Everything is loaded without a branch (absent tensors
// are empty buffers), so that one latency covers the lot.
// (48 sequences of one token, 5120 channels of 16 states: 8.6 us for 34 MB,
// 11.5 with branches between the loads, 24 in the tiled kernel)
template <typename T, int NPL, bool WHOLE>
__global__ __launch_bounds__(kThreads) void scan_step_kernel(ScanArgs a) {
  const int r = threadIdx.x & 3, g = blockIdx.z, Cg = a.G > 1 ? a.C / a.G : a.C;
  const int in = blockIdx.x * kChannels + (threadIdx.x >> 2);
  if (in >= Cg) return;
  const int c = g * Cg + in, b = blockIdx.y;
  Span sp = span_of(a.spans, b, a.T, a.rows);
  sp.first = __builtin_amdgcn_readfirstlane((int)sp.first);
  sp.len = __builtin_amdgcn_readfirstlane(sp.len);
  auto all = [](const void* p, int64_t offset, int64_t bytes) {
    return buffer_of(p, offset, p != nullptr ? bytes : 0);
  };
  const int64_t states = (int64_t)a.C * a.N * 4;  // at most 2^28
  const uint32_t oc = (uint32_t)c * a.N * 4u;
  float h[NPL], A[NPL];
  get_row<float, NPL, WHOLE>(all(a.S0, b * states, states), oc, r, a.N, h);
  get_row<float, NPL, WHOLE>(all(a.A, 0, states), oc, r, a.N, A);
  const float bias = get<float>(all(a.dt_bias, 0, a.C * 4), c * 4u);
  const float D = get<float>(all(a.D, 0, a.C * 4), c * 4u);
  for (int t = 0; t < sp.len; ++t) {
    const int64_t row = (sp.first + t) * (int64_t)sizeof(T);
    const uint32_t ot = c * (uint32_t)sizeof(T), on = g * a.N * (uint32_t)sizeof(T);
    const int64_t width = a.C * (int64_t)sizeof(T), bc = (int64_t)a.G * a.N * sizeof(T);
    float B[NPL], C[NPL];
    const float u = to_f32(get<T>(all(a.u, row * a.u_stride, width), ot));
    const float dt = to_f32(get<T>(all(a.dt, row * a.dt_stride, width), ot));
    const float z = to_f32(get<T>(all(a.z, row * a.z_stride, width), ot));
    get_row<T, NPL, WHOLE>(all(a.Bm, row * a.b_stride, bc), on, r, a.N, B);
    get_row<T, NPL, WHOLE>(all(a.Cm, row * a.c_stride, bc), on, r, a.N, C);
    if (t == 0 && a.ckpt != nullptr)
      put_states<NPL>(slot_buffer<NPL>(a.ckpt, slot_of(sp, b, save_steps<NPL>(), 0), a.C),
                      (uint32_t)(c * 4 * NPL + r * NPL) * 4u, h);
    // (log2 e goes to delta: to scale A first would wait for it before the
    // step's loads go out)
    const float dl = delta_of(dt + bias, a.softplus, true), du = dl * u, dl2 = kLog2e * dl;
    float acc = 0.f;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      // a step of delta = 0 changes nothing, at an infinite rate too (as
      // load_rates has it; here that would wait for A before the step's loads:
      // 48 tokens 8.24 us without, 8.32 so, 8.39 with it)
      const float e = dl2 == 0.f ? 0.f : dl2 * A[i];
      h[i] = fmaf(exp2_hw(e), h[i], du * B[i]);
      acc = fmaf(C[i], h[i], acc);
    }
    const float gate = silu(z);
    const float y = fmaf(D, u, quad_sum(acc)) * (a.z != nullptr ? gate : 1.f);
    put<T>(all(a.y, row * a.C, width), r == 0 ? ot : kNoLane, y);
  }
  if (a.S_T != nullptr)
    store_states<NPL>(a.S_T + ((int64_t)b * a.C + c) * a.N, a.N, r, true, h);
}

// The adjoint's first pass: E before the chunk (a_1 E_1 of its first step)
// from a zero E behind it, for every chunk but the first.
template <typename T, int NPL>
__global__ __launch_bounds__(kThreads)
SCAN_WAVES((NPL <= 8 ? 4 : 3)) void scan_adjoint_kernel(ScanArgs a, int ctiles) {
  constexpr int TT = tile_steps<NPL>();
  using L = Tile<T, NPL, TT, false, true, true>;
  constexpr int Q = L::Q, NP = L::NP;
  __shared__ __align__(16) float Cs[2][TT * NP];
  const Place p = place_of(a, ctiles);
  if (p.j > p.last) return;
  const int r = p.r;
  const uint32_t oh = p.cok ? (uint32_t)(p.c * NP + r * NPL) * 4u : kNoLane;
  if (p.j == 0) {
    if (p.last > 0) copy_start<NPL>(a, p, a.dS_T, 0, oh);
    return;
  }
  float A[NPL], E[NPL];
  load_rates<NPL>(a, p, A);
#pragma unroll
  for (int i = 0; i < NPL; ++i) E[i] = 0.f;
  const float bias = a.dt_bias != nullptr ? a.dt_bias[p.c] : 0.f;
  float sum = 0.f;
  L in;
  int t0 = p.begin + (p.end - p.begin - 1) / TT * TT;
  in.init(a, p, t0 - p.begin);
  typename L::Raw w;
  in.load(w);
  int buf = 0;
  for (; t0 >= p.begin; t0 -= TT, buf ^= 1) {
    float dl[Q], o[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      dl[q] = delta_of(to_f32(w.dt[q]) + bias, a.softplus, t0 + 4 * q + r < p.end);
      const float g = silu(to_f32(w.z[q]));
      o[q] = to_f32(w.dy[q]) * (a.z != nullptr ? g : 1.f);
      sum += dl[q];
    }
    L::stage(w, nullptr, Cs[buf]);
    in.template advance<-1>();
    if (t0 > p.begin) in.load(w);
    __syncthreads();
#pragma unroll
    for (int q = Q - 1; q >= 0; --q) {
      auto step = [&](auto kk) __attribute__((always_inline)) {
        constexpr int k = decltype(kk)::value;
        const float dk = quad_bcast<k>(dl[q]), ok_ = quad_bcast<k>(o[q]);
        const float* const cp = Cs[buf] + (4 * q + k) * NP + r * NPL;
#pragma unroll
        for (int i = 0; i < NPL; ++i) E[i] = exp2_hw(dk * A[i]) * fmaf(ok_, cp[i], E[i]);
      };
      step(std::integral_constant<int, 3>{});
      step(std::integral_constant<int, 2>{});
      step(std::integral_constant<int, 1>{});
      step(std::integral_constant<int, 0>{});
    }
  }
  const int64_t slot = slot_of(p.sp, p.b, a.chunk, p.j);
  put_states<NPL>(slot_buffer<NPL>(a.edge, slot, a.C), oh, E);
  sum = quad_sum(sum);
  if (r == 0 && p.cok) a.dsum[slot * a.C + p.c] = sum;
}

// The backward's main pass: tile by tile (of save_steps) the states are formed
// again from the saved one, with their decays, in registers, and the adjoint
// runs back over them.  One barrier a tile: the tile's B and C and its
// waves' parts of dB, dC sit in two buffers in turn, and a tile's parts are
// summed behind the next tile's barrier.
// WHOLE: every sequence ends with a tile.
template <typename T, int NPL, bool WHOLE>
__global__ __launch_bounds__(kThreads, (NPL <= 4 ? 3 : NPL <= 8 ? 2 : 1)) void scan_bwd_kernel(
    ScanArgs a, int ctiles) {
  constexpr int TT = save_steps<NPL>();
  using L = Tile<T, NPL, TT, true, true, true>;
  constexpr int NP = L::NP, Q = L::Q;
  __shared__ __align__(16) float Bs[2][TT * NP], Cs[2][TT * NP];
  __shared__ float red[2][kWaves][TT][2][NP];
  const Place p = place_of(a, ctiles);
  const int r = p.r, lane = threadIdx.x & 63;
  const uint32_t oh = p.cok ? (uint32_t)(p.c * NP + r * NPL) * 4u : kNoLane;
  // the place of its partial sums (formed here: in the end it would keep the
  // spans and sizes alive beside the tiles, 2% of the kernel), below 2^31
  // as it is at most one a row
  int place = (int)((int64_t)p.b * a.chunks + p.j);
  if (a.packed) {
    const int64_t at = pieces_before(a.spans, p.b, a.T, a.rows, a.chunk) + p.j;
    // (past the last: of sequences that overlap)
    place = p.j > p.last || p.sp.len == 0 || at >= a.parts ? -1 : (int)at;
    place = __builtin_amdgcn_readfirstlane(place);
  }
  float dA[NPL], sD = 0.f, sbias = 0.f;
#pragma unroll
  for (int i = 0; i < NPL; ++i) dA[i] = 0.f;
  if (p.j <= p.last) {
    float A[NPL], E[NPL];
    load_rates<NPL>(a, p, A);
    const float bias = a.dt_bias != nullptr ? a.dt_bias[p.c] : 0.f;
    const float D = a.D != nullptr ? a.D[p.c] : 0.f;
    start_states<NPL>(a, p, a.dS_T, 0, oh, E);
    join_chunks<false, NPL>(a, p, oh, A, E);
    const int tiles = (p.end - p.begin + TT - 1) / TT;
    int left = p.end - p.begin - (tiles - 1) * TT;  // steps of the tile at hand
    const int t_last = (tiles - 1) * TT;
    L in;
    in.init(a, p, tiles > 0 ? t_last : 0);
    typename L::Raw w;
    // the saved states, this channel tile's part of dB and dC, and the dense
    // gradients, with this lane's place in the tile at hand
    const int64_t steps = p.end - p.begin, row = p.sp.first + p.begin;
    const int64_t slot_bytes = (int64_t)a.C * NP * 4;
    const Buffer saved = buffer_of(a.ckpt, slot_of(p.sp, p.b, TT, p.begin / TT) * slot_bytes,
                                   tiles * slot_bytes);
    uint32_t osaved = oh + (tiles > 0 ? (uint32_t)(tiles - 1) * (uint32_t)slot_bytes : 0);
    const int64_t dense = row * (int64_t)in.sd, dense_bytes = steps * in.sd;
    const Buffer bdz = buffer_of(a.dz, dense, dense_bytes);
    const Buffer bdu = buffer_of(a.du, dense, dense_bytes);
    const Buffer bddt = buffer_of(a.ddt, dense, dense_bytes);
    const int tpg = ctiles / a.G;
    const uint32_t sbc = (uint32_t)(a.G * a.N) * 4u;
    const Buffer bdB =
        buffer_of(a.pB, ((int64_t)p.tile_in_group * a.rows + row) * sbc, steps * sbc);
    const Buffer bdC =
        buffer_of(a.pB, ((int64_t)(tpg + p.tile_in_group) * a.rows + row) * sbc, steps * sbc);
    const int bstep = threadIdx.x / NP, bn = threadIdx.x % NP;
    // (of the tile behind the one at hand: its parts are summed first)
    uint32_t obc = (uint32_t)(t_last + TT) * sbc +
                   (bn < a.N && bstep < TT ? bstep * sbc + (p.g * a.N + bn) * 4u : kNoLane);
    // dB, dC of the tile behind: the sum over the waves
    auto sum_waves = [&](int buf) __attribute__((always_inline)) {
      if (TT * NP < kThreads && bstep >= TT) return;
      float x = red[buf][0][bstep][0][bn], y = red[buf][0][bstep][1][bn];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) {
        x += red[buf][w][bstep][0][bn];
        y += red[buf][w][bstep][1][bn];
      }
      put<float>(bdB, obc, x);
      put<float>(bdC, obc, y);
    };
    float next[NPL];
    if (tiles > 0) {
      in.load(w);
      get_states<NPL>(saved, osaved, next);
    }
    int buf = 0;
    for (int tile = tiles - 1; tile >= 0; --tile, buf ^= 1) {
      // this lane's steps: delta and its slope, u, the gate's output and dy
      // times the gate's slope
      float dl[Q], slope[Q], u[Q], o[Q], dgate[Q], h0[NPL];
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const bool ok = 4 * q + r < left;
        const float raw = to_f32(w.dt[q]) + bias, sr = sigmoid(raw);
        u[q] = to_f32(w.u[q]);
        dl[q] = delta_of(raw, a.softplus, ok);
        slope[q] = ok ? (a.softplus ? sr : 1.f) : 0.f;
        const float dy = to_f32(w.dy[q]), z = to_f32(w.z[q]), sg = sigmoid(z);
        dgate[q] = dy * dsilu(z, sg);
        o[q] = dy * (a.z != nullptr ? z * sg : 1.f);
        sD = fmaf(o[q], u[q], sD);
      }
#pragma unroll
      for (int i = 0; i < NPL; ++i) h0[i] = next[i];
      L::stage(w, Bs[buf], Cs[buf]);
      const uint32_t dense_at = in.od;
      in.template advance<-1>();
      osaved -= (uint32_t)slot_bytes;
      if (tile > 0) {
        in.load(w);
        get_states<NPL>(saved, osaved, next);
      }
      __syncthreads();
      if (tile < tiles - 1) sum_waves(buf ^ 1);
      obc -= TT * sbc;
      float h[TT][NPL], dec[TT][NPL];
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const float du = dl[q] * u[q];
        float acc[4];
        auto step = [&](auto kk) __attribute__((always_inline)) {
          constexpr int e = decltype(kk)::value;
          const int s = 4 * q + e;
          const float dk = quad_bcast<e>(dl[q]), duk = quad_bcast<e>(du);
          const float* const bp = Bs[buf] + s * NP + r * NPL;
          const float* const cp = Cs[buf] + s * NP + r * NPL;
          acc[e] = 0.f;
#pragma unroll
          for (int i = 0; i < NPL; ++i) {
            const float prev = s > 0 ? h[s > 0 ? s - 1 : 0][i] : h0[i];
            dec[s][i] = exp2_hw(dk * A[i]);
            h[s][i] = fmaf(dec[s][i], prev, duk * bp[i]);
            acc[e] = fmaf(cp[i], h[s][i], acc[e]);
          }
        };
        step(std::integral_constant<int, 0>{});
        step(std::integral_constant<int, 1>{});
        step(std::integral_constant<int, 2>{});
        step(std::integral_constant<int, 3>{});
        if (a.z != nullptr) {
          const float read = fmaf(D, u[q], quad_scatter_sum(acc, r));
          put<T>(bdz, dense_at + 4 * q * in.sd, dgate[q] * read);
        }
      }
#pragma unroll
      for (int q = Q - 1; q >= 0; --q) {
        const float du = dl[q] * u[q];
        float sB[4], sA[4];
        auto step = [&](auto kk) __attribute__((always_inline)) {
          constexpr int e = decltype(kk)::value;
          constexpr int NH = NPL > 1 ? NPL / 2 : 1;
          const int s = 4 * q + e;
          const float dk = quad_bcast<e>(dl[q]), duk = quad_bcast<e>(du);
          const float o_ = quad_bcast<e>(o[q]);
          const float* const bp = Bs[buf] + s * NP + r * NPL;
          const float* const cp = Cs[buf] + s * NP + r * NPL;
          float v[2 * NPL];
          sB[e] = sA[e] = 0.f;
          // A step past the end passes E on and adds nothing.  It is skipped:
          // its delta and slope of 0 times an infinite rate, state or product
          // would be NaN in dA and ddt_bias.  (A branch the whole wave takes;
          // masks, or a form of their own for last tiles, push the kernel past
          // its registers: 1480 us at 4 x 4096 x 4096.)
          if (!WHOLE && s > 0 && s >= left) return;
#pragma unroll
          for (int i = 0; i < NPL; ++i) {
            const float prev = s > 0 ? h[s > 0 ? s - 1 : 0][i] : h0[i];
            const float ad = fmaf(o_, cp[i], E[i]);
            v[i] = ad * duk;
            v[NPL + i] = o_ * h[s][i];
            sB[e] = fmaf(ad, bp[i], sB[e]);
            E[i] = ad * dec[s][i];
            const float m = E[i] * prev;
            sA[e] = fmaf(A[i], m, sA[e]);
            dA[i] = fmaf(dk, m, dA[i]);
          }
          float w[NH];
          quads_scatter_sum<2 * NPL>(v, w);
          // values NH (l / 16) .. of [dB | dC]: row l / 32, states from
          // r NPL + NH (l / 16 % 2)
          const int odd = NPL > 1 ? (lane >> 4) & 1 : 0;
          if ((lane & 12) == 0)
#pragma unroll
            for (int i = 0; i < NH; ++i)
              red[buf][p.wave][s][lane >> 5][r * NPL + odd * NH + i] = w[i];
        };
        step(std::integral_constant<int, 3>{});
        step(std::integral_constant<int, 2>{});
        step(std::integral_constant<int, 1>{});
        step(std::integral_constant<int, 0>{});
        const float gB = quad_scatter_sum(sB, r);
        const float gA = kLn2 * quad_scatter_sum(sA, r);  // A holds log2(e) A
        const float ddt = fmaf(u[q], gB, gA) * slope[q];
        const uint32_t to = dense_at + 4 * q * in.sd;
        put<T>(bdu, to, fmaf(D, o[q], dl[q] * gB));
        put<T>(bddt, to, ddt);
        sbias += ddt;
      }
      left = TT;
    }
    __syncthreads();
    if (tiles > 0) sum_waves(buf ^ 1);
    if (p.j == 0 && a.dS0 != nullptr)
      store_states<NPL>(a.dS0 + ((int64_t)p.b * a.C + p.c) * a.N, a.N, r, p.cok, E);
  }
  // partial dA, dD and ddt_bias: zeros from a chunk without steps, or none
  // where they are numbered through the chunks that have some
  if (place < 0) return;
  float* const part = a.pA + (int64_t)place * a.C * (NP + 2);
  put_states<NPL>(buffer_of(part, 0, (int64_t)a.C * NP * 4), oh, dA);
  sD = quad_sum(sD);
  sbias = quad_sum(sbias);
  if (r == 0 && p.cok) {
    part[(int64_t)a.C * NP + p.c] = sD;
    part[(int64_t)a.C * (NP + 1) + p.c] = sbias;
  }
}

// The backward's sums, in one launch: workgroups [0, ca) of sequence 0 sum
// the chunks' partial dA, dD, ddt_bias, 16 columns and 16 chunk lanes each;
// the others sum dB, dC of their sequence's rows over the channel tiles.
struct SumGrid {
  int ca, tpg, NP;
};
template <typename T>
__global__ __launch_bounds__(kThreads) void scan_sums(ScanArgs a, SumGrid g) {
  if ((int)blockIdx.x < g.ca) {
    if (blockIdx.y > 0) return;
    const int64_t width = (int64_t)a.C * (g.NP + 2);
    const int64_t i = (int64_t)blockIdx.x * kSumCols + threadIdx.x % kSumCols;
    int64_t parts = a.parts;
    if (a.packed) {
      const int64_t used = pieces_before(a.spans, a.B, a.T, a.rows, a.chunk);
      parts = used < parts ? used : parts;
    }
    const float x = column_sum(a.pA, parts, width, i);
    if (threadIdx.x >= kSumCols || i >= width) return;
    if (i < (int64_t)a.C * g.NP) {
      const int64_t c = i / g.NP, n = i % g.NP;
      if (n < a.N) a.dA[c * a.N + n] = x;
    } else if (i < (int64_t)a.C * (g.NP + 1)) {
      if (a.dD != nullptr) a.dD[i - (int64_t)a.C * g.NP] = x;
    } else if (a.ddt_bias != nullptr) {
      a.ddt_bias[i - (int64_t)a.C * (g.NP + 1)] = x;
    }
    return;
  }
  const Span sp = span_of(a.spans, blockIdx.y, a.T, a.rows);
  const int64_t w = (int64_t)a.G * a.N, all = a.rows * w;
  const int64_t turn = (int64_t)(gridDim.x - g.ca) * kThreads;
  for (int64_t i = (int64_t)(blockIdx.x - g.ca) * kThreads + threadIdx.x; i < w * sp.len;
       i += turn) {
    const int64_t at = sp.first * w + i;
    float sb = 0.f, sc = 0.f;
#pragma unroll 4
    for (int k = 0; k < g.tpg; ++k) {
      sb += a.pB[k * all + at];
      sc += a.pB[(g.tpg + k) * all + at];
    }
    st(static_cast<T*>(a.dB), at, sb);
    st(static_cast<T*>(a.dC), at, sc);
  }
}

hipError_t noted(hipStream_t s) {
  const hipError_t e = hipGetLastError();
  note_launch(s);
  return e;
}

int channel_tiles(int64_t C, int64_t G) {
  return (int)(G * ((C / G + kChannels - 1) / kChannels));
}

template <typename T, int NPL>
hipError_t fwd(const ScanArgs& a, hipStream_t s) {
  const int ct = channel_tiles(a.C, a.G);
  if (a.T <= kMaxStep) {
    const dim3 grid((unsigned)(ct / a.G), a.B, a.G);
    if (a.N == 4 * NPL && a.b_stride % 4 == 0 && a.c_stride % 4 == 0)
      hipLaunchKernelGGL((scan_step_kernel<T, NPL, true>), grid, dim3(kThreads), 0, s, a);
    else
      hipLaunchKernelGGL((scan_step_kernel<T, NPL, false>), grid, dim3(kThreads), 0, s, a);
    return noted(s);
  }
  const dim3 grid((unsigned)(ct * a.chunks), a.B);
  hipError_t e;
  if (a.chunks > 1) {
    hipLaunchKernelGGL((scan_fwd_kernel<T, NPL, true>), grid, dim3(kThreads), 0, s, a, ct);
    if ((e = noted(s)) != hipSuccess) return e;
  }
  hipLaunchKernelGGL((scan_fwd_kernel<T, NPL, false>), grid, dim3(kThreads), 0, s, a, ct);
  return noted(s);
}

template <typename T, int NPL>
hipError_t bwd(const ScanArgs& a, hipStream_t s) {
  const int ct = channel_tiles(a.C, a.G), np = 4 * NPL;
  const dim3 grid((unsigned)(ct * a.chunks), a.B);
  hipError_t e;
  if (a.chunks > 1) {
    hipLaunchKernelGGL((scan_adjoint_kernel<T, NPL>), grid, dim3(kThreads), 0, s, a, ct);
    if ((e = noted(s)) != hipSuccess) return e;
  }
  // The branch around padding steps costs a backward pass of 4 x 4096 x 4096
  // with 16 states 20 us (985 -> 1005), of 2048 x 4096 with 32 states 5 (250 ->
  // 255), with fewer states nothing; with 64 states it gains (630 -> 602, fewer
  // registers alive).
  if ((NPL == 4 || NPL == 8) && a.spans == nullptr && a.T % save_steps<NPL>() == 0)
    hipLaunchKernelGGL((scan_bwd_kernel<T, NPL, NPL == 4 || NPL == 8>), grid, dim3(kThreads), 0, s,
                       a, ct);
  else
    hipLaunchKernelGGL((scan_bwd_kernel<T, NPL, false>), grid, dim3(kThreads), 0, s, a, ct);
  if ((e = noted(s)) != hipSuccess) return e;
  const int64_t columns = (int64_t)a.C * (np + 2), values = (int64_t)a.T * a.G * a.N;
  const SumGrid g{(int)((columns + kSumCols - 1) / kSumCols), ct / a.G, np};
  int64_t blocks = g.ca + (values + kThreads - 1) / kThreads;
  if (blocks > kMaxGrid) blocks = kMaxGrid;  // (ca is at most 2^20 66 / 16)
  hipLaunchKernelGGL((scan_sums<T>), dim3((unsigned)blocks, a.B), dim3(kThreads), 0, s, a, g);
  return noted(s);
}

template <typename T, bool BWD>
hipError_t launch(const ScanArgs& a, hipStream_t s) {
  switch (scan_padded(a.N)) {
    case 4: return BWD ? bwd<T, 1>(a, s) : fwd<T, 1>(a, s);
    case 8: return BWD ? bwd<T, 2>(a, s) : fwd<T, 2>(a, s);
    case 16: return BWD ? bwd<T, 4>(a, s) : fwd<T, 4>(a, s);
    case 32: return BWD ? bwd<T, 8>(a, s) : fwd<T, 8>(a, s);
    case 64: return BWD ? bwd<T, 16>(a, s) : fwd<T, 16>(a, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace

int scan_padded(int64_t N) { return N <= 4 ? 4 : N <= 8 ? 8 : N <= 16 ? 16 : N <= 32 ? 32 : 64; }
int scan_save_steps(int64_t N) { return N <= 16 ? 8 : 4; }
int scan_channels() { return kChannels; }

int64_t scan_chunk(const ScanArgs& a, int64_t stride, bool bwd) {
  const int64_t T = a.T;
  if (a.B == 0 || T == 0) return 16;
  // Waves of the unsplit grid; packed sequences count for their rows.
  // Measured at C = 4096, N = 16, bf16, forward / backward in us, by chunks:
  //    256 waves (T = 2048)  1: 236 / 588   8: 91 / 168   16: 83 / 153   32: 88 / 157
  //    512                   1: 238 / 598   8: 161 / 304  16: 161 / 309
  //   1024 (T = 4096)        1: 449 / 1181  3: 537 / 1043  8: 535 / 1006  16: 547 / 1031
  //   2048 (T = 2048)        1: 390 / 891   2: 552 / 1043  8: 531 / 1022
  // A chunk more than one repeats most of the recurrence in the first pass,
  // which pays while the device has waves missing: below one wave a SIMD
  // forward, two backward (its main pass waits more).  Then 4096 waves or more,
  // and chunks of at least 32 steps; joining bounds their number.
  const int64_t waves = a.rows * channel_tiles(a.C, a.G) * kWaves / T;
  int64_t S = 1;
  if (waves < (bwd ? 2048 : 1024)) {
    S = 4096 / (waves > 0 ? waves : 1);
    S = S < 8 ? 8 : (S > kMaxChunks ? kMaxChunks : S);
  }
  int64_t L = (T + S - 1) / S;
  if (L < 32) L = 32 < T ? 32 : T;
  L = (L + 15) / 16 * 16;
  // the most steps whose rows and saved states stay below 2^31 bytes
  const int64_t row = 4 * stride;
  const int64_t state = 4 * (int64_t)a.C * scan_padded(a.N) / scan_save_steps(a.N);
  const int64_t most = (INT64_C(1) << 31) / (row > state ? row : state) / 16 * 16;
  return L < most ? L : most;
}

hipError_t launch_scan_fwd(const ScanArgs& a, bool is_bf16, hipStream_t s) {
  return is_bf16 ? launch<bf16, false>(a, s) : launch<float, false>(a, s);
}
hipError_t launch_scan_bwd(const ScanArgs& a, bool is_bf16, hipStream_t s) {
  return is_bf16 ? launch<bf16, true>(a, s) : launch<float, true>(a, s);
}

}  // namespace gdr
