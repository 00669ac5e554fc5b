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
// Every state and step takes one exponential (a quarter-rate instruction)
// and 4 (forward) or 12 (backward) products and sums: bound by the vector
// units, not by HBM.
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
// start (edge) and its sum of delta (dsum), scan_join turns those into the
// state before every chunk, h_in(j + 1) = exp(A dsum_j) h_in(j) + edge_j, and
// the main pass starts from them.  The backward joins the adjoint the same
// way.
#include "gdr_layer.h"

namespace gdr {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kChannels = 64;  // of one workgroup

template <int NPL>
constexpr int tile_steps() {
  return NPL <= 4 ? 16 : 64 / NPL;
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
__device__ __forceinline__ float swap32_sum(float a, float b) {
  const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false,
                                                  false);
  return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}
__device__ __forceinline__ float swap16_sum(float a, float b) {
  const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false,
                                                  false);
  return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}
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
__device__ __forceinline__ Place place_of(const ScanArgs& a, int ctiles) {
  Place p;
  p.b = blockIdx.y;
  p.sp = span_of(a.spans, p.b, a.T, a.rows);
  const int ct = blockIdx.x % ctiles, tpg = ctiles / a.G;
  p.j = blockIdx.x / ctiles;
  p.g = ct / tpg;
  p.tile_in_group = ct % tpg;
  p.wave = threadIdx.x >> 6;
  p.r = threadIdx.x & 3;
  const int Cg = a.C / a.G;
  const int in = p.tile_in_group * kChannels + (threadIdx.x >> 2);
  p.cok = in < Cg;
  p.c = p.g * Cg + (p.cok ? in : 0);
  p.last = p.sp.len > 0 ? (p.sp.len - 1) / a.chunk : 0;
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

template <int NPL>
__device__ __forceinline__ void load_states(const float* p, int N, int r, bool ok,
                                            float (&h)[NPL]) {
#pragma unroll
  for (int i = 0; i < NPL; ++i) h[i] = ok && r * NPL + i < N ? p[r * NPL + i] : 0.f;
}
template <int NPL>
__device__ __forceinline__ void store_states(float* p, int N, int r, bool ok,
                                             const float (&h)[NPL]) {
#pragma unroll
  for (int i = 0; i < NPL; ++i)
    if (ok && r * NPL + i < N) p[r * NPL + i] = h[i];
}
// The same for buffers with 4 NPL states per channel: whole vectors.
template <int NPL>
struct alignas(NPL >= 4 ? 16 : 4 * NPL) States {
  float v[NPL];
};

// The raw loads of one tile: this lane's steps of its channel, and this
// thread's element of B and C.  Steps past the end read the last one.
template <typename T, int NPL, bool IN, bool OUT>
struct Tile {
  static constexpr int TT = tile_steps<NPL>(), Q = TT / 4, NP = 4 * NPL;
  T u[Q], dt[Q], z[Q], dy[Q];
  T bm, cm;

  __device__ __forceinline__ void load(const ScanArgs& a, const Place& p, int t0, bool with_dy) {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      int t = t0 + 4 * q + p.r;
      t = t < p.sp.len ? t : p.sp.len - 1;
      const int64_t row = p.sp.first + t;
      if (IN) u[q] = static_cast<const T*>(a.u)[row * a.u_stride + p.c];
      dt[q] = static_cast<const T*>(a.dt)[row * a.dt_stride + p.c];
      if (OUT && a.z != nullptr) z[q] = static_cast<const T*>(a.z)[row * a.z_stride + p.c];
      if (OUT && with_dy) dy[q] = static_cast<const T*>(a.dy)[row * a.C + p.c];
    }
    const int i = threadIdx.x;
    int t = t0 + i / NP;
    t = t < p.sp.len ? t : p.sp.len - 1;
    const int n = i % NP < a.N ? i % NP : 0;
    const int64_t row = p.sp.first + t;
    if (IN) bm = static_cast<const T*>(a.Bm)[row * a.b_stride + (int64_t)p.g * a.N + n];
    if (OUT) cm = static_cast<const T*>(a.Cm)[row * a.c_stride + (int64_t)p.g * a.N + n];
  }
  // B and C to LDS, zeros in the padding and past the end
  __device__ __forceinline__ void stage(const ScanArgs& a, const Place& p, int t0, float* bs,
                                        float* cs) const {
    const int i = threadIdx.x;
    if (i >= TT * NP) return;
    const bool ok = t0 + i / NP < p.sp.len && i % NP < a.N;
    if (IN) bs[i] = ok ? to_f32(bm) : 0.f;
    if (OUT) cs[i] = ok ? to_f32(cm) : 0.f;
  }
};

// delta of a raw step; 0, an identity step, outside the sequence.
__device__ __forceinline__ float delta_of(float raw, int plus, bool ok) {
  const float d = plus ? softplus(raw) : raw;
  return ok ? d : 0.f;
}

template <int NPL>
__device__ __forceinline__ void load_rates(const ScanArgs& a, const Place& p, float (&A)[NPL]) {
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int n = p.r * NPL + i;
    A[i] = p.cok && n < a.N ? kLog2e * a.A[(int64_t)p.c * a.N + n] : 0.f;
  }
}

// EDGE: the first pass (end state of every chunk but the last from a zero
// start); else the pass that writes y.
template <typename T, int NPL, bool EDGE>
__global__ __launch_bounds__(kThreads) void scan_fwd_kernel(ScanArgs a, int ctiles) {
  using L = Tile<T, NPL, true, !EDGE>;
  constexpr int TT = L::TT, Q = L::Q, NP = L::NP;
  __shared__ __align__(16) float Bs[2][TT * NP], Cs[2][EDGE ? 4 : TT * NP];
  const Place p = place_of(a, ctiles);
  if (EDGE ? p.j >= p.last : p.j > p.last) return;
  const int r = p.r;
  float A[NPL], h[NPL];
  load_rates<NPL>(a, p, A);
  const float bias = a.dt_bias != nullptr ? a.dt_bias[p.c] : 0.f;
  const float D = a.D != nullptr ? a.D[p.c] : 0.f;
  float* const edge = a.chunks > 1 ? a.edge + (slot_of(p.sp, p.b, a.chunk, p.j) * a.C + p.c) * NP
                                   : nullptr;
  if (EDGE) {
#pragma unroll
    for (int i = 0; i < NPL; ++i) h[i] = 0.f;
  } else if (a.chunks > 1) {
    const States<NPL> s = *reinterpret_cast<const States<NPL>*>(edge + r * NPL);
#pragma unroll
    for (int i = 0; i < NPL; ++i) h[i] = s.v[i];
  } else {
    load_states<NPL>(a.S0 + ((int64_t)p.b * a.C + p.c) * a.N, a.N, r, p.cok && a.S0 != nullptr, h);
  }
  float sum = 0.f;
  L in;
  if (p.begin < p.end) in.load(a, p, p.begin, false);
  int buf = 0;
  for (int t0 = p.begin; t0 < p.end; t0 += TT, buf ^= 1) {
    in.stage(a, p, t0, Bs[buf], Cs[buf]);
    __syncthreads();
    const L cur = in;
    if (t0 + TT < p.end) in.load(a, p, t0 + TT, false);
    if (!EDGE && a.ckpt != nullptr && p.cok) {
      States<NPL> s;
#pragma unroll
      for (int i = 0; i < NPL; ++i) s.v[i] = h[i];
      *reinterpret_cast<States<NPL>*>(
          a.ckpt + (slot_of(p.sp, p.b, TT, t0 / TT) * a.C + p.c) * NP + r * NPL) = s;
    }
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int t = t0 + 4 * q + r;
      const bool ok = p.cok && t < p.end;
      const float u = to_f32(cur.u[q]);
      const float dl = delta_of(to_f32(cur.dt[q]) + bias, a.softplus, ok);
      const float du = ok ? dl * u : 0.f;
      sum += dl;
      float acc[4];
      auto step = [&](auto kk) __attribute__((always_inline)) {
        constexpr int k = decltype(kk)::value;
        const float dk = quad_bcast<k>(dl), duk = quad_bcast<k>(du);
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
        float y = fmaf(D, u, quad_scatter_sum(acc, r));
        if (a.z != nullptr) y *= silu(to_f32(cur.z[q]));
        if (ok) st(static_cast<T*>(a.y), (p.sp.first + t) * a.C + p.c, y);
      }
    }
  }
  if (EDGE) {
    if (!p.cok) return;
    States<NPL> s;
#pragma unroll
    for (int i = 0; i < NPL; ++i) s.v[i] = h[i];
    *reinterpret_cast<States<NPL>*>(edge + r * NPL) = s;
    sum = quad_sum(sum);
    if (r == 0) a.dsum[slot_of(p.sp, p.b, a.chunk, p.j) * a.C + p.c] = sum;
  } else if (p.j == p.last && a.S_T != nullptr) {
    store_states<NPL>(a.S_T + ((int64_t)p.b * a.C + p.c) * a.N, a.N, r, p.cok, h);
  }
}

// The adjoint's first pass: E before the chunk (a_1 E_1 of its first step)
// from a zero E behind it, for every chunk but the first.
template <typename T, int NPL>
__global__ __launch_bounds__(kThreads) void scan_adjoint_kernel(ScanArgs a, int ctiles) {
  using L = Tile<T, NPL, false, true>;
  constexpr int TT = L::TT, Q = L::Q, NP = L::NP;
  __shared__ __align__(16) float Cs[2][TT * NP];
  const Place p = place_of(a, ctiles);
  if (p.j == 0 || p.j > p.last) return;
  const int r = p.r;
  float A[NPL], E[NPL];
  load_rates<NPL>(a, p, A);
#pragma unroll
  for (int i = 0; i < NPL; ++i) E[i] = 0.f;
  const float bias = a.dt_bias != nullptr ? a.dt_bias[p.c] : 0.f;
  float sum = 0.f;
  L in;
  int t0 = p.begin + (p.end - p.begin - 1) / TT * TT;
  in.load(a, p, t0, true);
  int buf = 0;
  for (; t0 >= p.begin; t0 -= TT, buf ^= 1) {
    in.stage(a, p, t0, nullptr, Cs[buf]);
    __syncthreads();
    const L cur = in;
    if (t0 > p.begin) in.load(a, p, t0 - TT, true);
#pragma unroll
    for (int q = Q - 1; q >= 0; --q) {
      const bool ok = p.cok && t0 + 4 * q + r < p.end;
      const float dl = delta_of(to_f32(cur.dt[q]) + bias, a.softplus, ok);
      float o = to_f32(cur.dy[q]);
      if (a.z != nullptr) o *= silu(to_f32(cur.z[q]));
      o = ok ? o : 0.f;
      sum += dl;
      auto step = [&](auto kk) __attribute__((always_inline)) {
        constexpr int k = decltype(kk)::value;
        const float dk = quad_bcast<k>(dl), ok_ = quad_bcast<k>(o);
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
  if (!p.cok) return;
  const int64_t slot = slot_of(p.sp, p.b, a.chunk, p.j);
  States<NPL> s;
#pragma unroll
  for (int i = 0; i < NPL; ++i) s.v[i] = E[i];
  *reinterpret_cast<States<NPL>*>(a.edge + (slot * a.C + p.c) * NP + r * NPL) = s;
  sum = quad_sum(sum);
  if (r == 0) a.dsum[slot * a.C + p.c] = sum;
}

// Turns the chunks' local end states into the state before every chunk
// (FWD), or the local adjoints into the adjoint behind every chunk.  One
// thread per channel and padded state; four chunks' loads in flight.
template <bool FWD>
__global__ __launch_bounds__(kThreads) void scan_join_kernel(ScanArgs a, int NP) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= (int64_t)a.C * NP) return;
  const int b = blockIdx.y;
  const Span sp = span_of(a.spans, b, a.T, a.rows);
  const int last = sp.len > 0 ? (sp.len - 1) / a.chunk : 0;
  const int c = (int)(i / NP), n = (int)(i % NP);
  const bool ok = n < a.N;
  const float A = ok ? kLog2e * a.A[(int64_t)c * a.N + n] : 0.f;
  const float* const start = FWD ? a.S0 : a.dS_T;
  float h = ok && start != nullptr ? start[((int64_t)b * a.C + c) * a.N + n] : 0.f;
  const int64_t s0 = slot_of(sp, b, a.chunk, 0), stride = (int64_t)a.C * NP;
  constexpr int U = 4;
  for (int k0 = 0; k0 <= last; k0 += U) {
    float e[U], d[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      // chunks in the order of the recurrence; the one at its end has no edge
      const bool has = k0 + k < last;
      const int64_t s = s0 + (has ? (FWD ? k0 + k : last - k0 - k) : (FWD ? 0 : last));
      e[k] = a.edge[s * stride + i];
      d[k] = a.dsum[s * a.C + c];
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (k0 + k > last) break;
      a.edge[(s0 + (FWD ? k0 + k : last - k0 - k)) * stride + i] = h;
      if (k0 + k < last) h = fmaf(exp2_hw(A * d[k]), h, e[k]);
    }
  }
}

// The backward's main pass: per tile the states are formed again from the
// saved one, with the decays kept in registers, and the adjoint runs back
// over them.
template <typename T, int NPL>
__global__ __launch_bounds__(kThreads, 2) void scan_bwd_kernel(ScanArgs a, int ctiles) {
  using L = Tile<T, NPL, true, true>;
  constexpr int TT = L::TT, Q = L::Q, NP = L::NP;
  __shared__ __align__(16) float Bs[TT * NP], Cs[TT * NP];
  __shared__ float red[kWaves][TT][2][NP];
  const Place p = place_of(a, ctiles);
  const int r = p.r, lane = threadIdx.x & 63;
  float dA[NPL], sD = 0.f, sbias = 0.f;
#pragma unroll
  for (int i = 0; i < NPL; ++i) dA[i] = 0.f;
  if (p.j <= p.last) {
    float A[NPL], E[NPL];
    load_rates<NPL>(a, p, A);
    const float bias = a.dt_bias != nullptr ? a.dt_bias[p.c] : 0.f;
    const float D = a.D != nullptr ? a.D[p.c] : 0.f;
    if (a.chunks > 1) {
      const States<NPL> s = *reinterpret_cast<const States<NPL>*>(
          a.edge + (slot_of(p.sp, p.b, a.chunk, p.j) * a.C + p.c) * NP + r * NPL);
#pragma unroll
      for (int i = 0; i < NPL; ++i) E[i] = p.cok ? s.v[i] : 0.f;
    } else {
      load_states<NPL>(a.dS_T + ((int64_t)p.b * a.C + p.c) * a.N, a.N, r,
                       p.cok && a.dS_T != nullptr, E);
    }
    L in;
    const int tiles = (p.end - p.begin + TT - 1) / TT;
    int t0 = p.begin + (tiles - 1) * TT;
    if (tiles > 0) in.load(a, p, t0, true);
    const int tpg = ctiles / a.G;
    for (int tile = tiles - 1; tile >= 0; --tile, t0 -= TT) {
      in.stage(a, p, t0, Bs, Cs);
      __syncthreads();
      const L cur = in;
      if (tile > 0) in.load(a, p, t0 - TT, true);
      float h0[NPL];
      {
        const States<NPL> s = *reinterpret_cast<const States<NPL>*>(
            a.ckpt + (slot_of(p.sp, p.b, TT, t0 / TT) * a.C + p.c) * NP + r * NPL);
#pragma unroll
        for (int i = 0; i < NPL; ++i) h0[i] = p.cok ? s.v[i] : 0.f;
      }
      float dl[Q], u[Q], o[Q], h[TT][NPL], dec[TT][NPL];
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const int t = t0 + 4 * q + r;
        const bool ok = p.cok && t < p.end;
        u[q] = ok ? to_f32(cur.u[q]) : 0.f;
        dl[q] = delta_of(to_f32(cur.dt[q]) + bias, a.softplus, ok);
        const float du = dl[q] * u[q];
        float acc[4];
        auto step = [&](auto kk) __attribute__((always_inline)) {
          constexpr int k = decltype(kk)::value;
          const float dk = quad_bcast<k>(dl[q]), duk = quad_bcast<k>(du);
          const float* const bp = Bs + (4 * q + k) * NP + r * NPL;
          const float* const cp = Cs + (4 * q + k) * NP + r * NPL;
          acc[k] = 0.f;
#pragma unroll
          for (int i = 0; i < NPL; ++i) {
            const float prev = 4 * q + k > 0 ? h[4 * q + k > 0 ? 4 * q + k - 1 : 0][i] : h0[i];
            dec[4 * q + k][i] = exp2_hw(dk * A[i]);
            h[4 * q + k][i] = fmaf(dec[4 * q + k][i], prev, duk * bp[i]);
            acc[k] = fmaf(cp[i], h[4 * q + k][i], acc[k]);
          }
        };
        step(std::integral_constant<int, 0>{});
        step(std::integral_constant<int, 1>{});
        step(std::integral_constant<int, 2>{});
        step(std::integral_constant<int, 3>{});
        o[q] = to_f32(cur.dy[q]);
        if (a.z != nullptr) {
          const float z = to_f32(cur.z[q]), sg = sigmoid(z);
          const float read = fmaf(D, u[q], quad_scatter_sum(acc, r));
          if (ok)
            st(static_cast<T*>(a.dz), (p.sp.first + t) * a.C + p.c, o[q] * read * dsilu(z, sg));
          o[q] *= z * sg;
        }
        o[q] = ok ? o[q] : 0.f;
        sD = fmaf(o[q], u[q], sD);
      }
#pragma unroll
      for (int q = Q - 1; q >= 0; --q) {
        const int t = t0 + 4 * q + r;
        const bool ok = p.cok && t < p.end;
        const float du = dl[q] * u[q];
        float sB[4], sA[4];
        auto step = [&](auto kk) __attribute__((always_inline)) {
          constexpr int k = decltype(kk)::value;
          constexpr int NH = NPL > 1 ? NPL / 2 : 1;
          const int s = 4 * q + k;
          const float dk = quad_bcast<k>(dl[q]), duk = quad_bcast<k>(du), o_ = quad_bcast<k>(o[q]);
          const float* const bp = Bs + s * NP + r * NPL;
          const float* const cp = Cs + s * NP + r * NPL;
          float v[2 * NPL];
          sB[k] = sA[k] = 0.f;
#pragma unroll
          for (int i = 0; i < NPL; ++i) {
            const float prev = s > 0 ? h[s > 0 ? s - 1 : 0][i] : h0[i];
            const float e = fmaf(o_, cp[i], E[i]);
            v[i] = e * duk;
            v[NPL + i] = o_ * h[s][i];
            sB[k] = fmaf(e, bp[i], sB[k]);
            E[i] = e * dec[s][i];
            const float m = E[i] * prev;
            sA[k] = fmaf(A[i], m, sA[k]);
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
              red[p.wave][s][lane >> 5][r * NPL + odd * NH + i] = w[i];
        };
        step(std::integral_constant<int, 3>{});
        step(std::integral_constant<int, 2>{});
        step(std::integral_constant<int, 1>{});
        step(std::integral_constant<int, 0>{});
        const float gB = quad_scatter_sum(sB, r);
        const float gA = kLn2 * quad_scatter_sum(sA, r);  // A holds log2(e) A
        float ddt = fmaf(u[q], gB, gA);
        if (a.softplus) ddt *= sigmoid(to_f32(cur.dt[q]) + bias);
        if (ok) {
          const int64_t at = (p.sp.first + t) * a.C + p.c;
          st(static_cast<T*>(a.du), at, fmaf(D, o[q], dl[q] * gB));
          st(static_cast<T*>(a.ddt), at, ddt);
          sbias += ddt;
        }
      }
      __syncthreads();
      for (int i = threadIdx.x; i < 2 * TT * NP; i += kThreads) {
        const int which = i / (TT * NP), s = i / NP % TT, n = i % NP;
        if (t0 + s < p.end && n < a.N) {
          float x = red[0][s][which][n];
#pragma unroll
          for (int w = 1; w < kWaves; ++w) x += red[w][s][which][n];
          a.pB[(((int64_t)which * tpg + p.tile_in_group) * a.rows + p.sp.first + t0 + s) * a.G *
                   a.N +
               (int64_t)p.g * a.N + n] = x;
        }
      }
    }
    if (p.j == 0 && a.dS0 != nullptr)
      store_states<NPL>(a.dS0 + ((int64_t)p.b * a.C + p.c) * a.N, a.N, r, p.cok, E);
  }
  if (!p.cok) return;
  // partial dA, dD and ddt_bias: zeros from a chunk without steps
  float* const part = a.pA + ((int64_t)p.b * a.chunks + p.j) * a.C * (NP + 2);
  States<NPL> s;
#pragma unroll
  for (int i = 0; i < NPL; ++i) s.v[i] = dA[i];
  *reinterpret_cast<States<NPL>*>(part + (int64_t)p.c * NP + r * NPL) = s;
  sD = quad_sum(sD);
  sbias = quad_sum(sbias);
  if (r == 0) {
    part[(int64_t)a.C * NP + p.c] = sD;
    part[(int64_t)a.C * (NP + 1) + p.c] = sbias;
  }
}

// dB, dC of every row of a sequence: the sums over the channel tiles.
template <typename T>
__global__ __launch_bounds__(kThreads) void scan_sum_bc(ScanArgs a, int tpg) {
  const Span sp = span_of(a.spans, blockIdx.y, a.T, a.rows);
  const int64_t w = (int64_t)a.G * a.N;
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= w * sp.len) return;
  const int64_t at = sp.first * w + i, all = a.rows * w;
  float sb = 0.f, sc = 0.f;
#pragma unroll 4
  for (int k = 0; k < tpg; ++k) {
    sb += a.pB[k * all + at];
    sc += a.pB[(tpg + k) * all + at];
  }
  st(static_cast<T*>(a.dB), at, sb);
  st(static_cast<T*>(a.dC), at, sc);
}

struct ScanSumStore {
  float* dA;
  float* dD;
  float* ddt_bias;
  int C, N, NP;
  __device__ void operator()(int64_t i, float x) const {
    if (i < (int64_t)C * NP) {
      const int64_t c = i / NP, n = i % NP;
      if (n < N) dA[c * N + n] = x;
    } else if (i < (int64_t)C * (NP + 1)) {
      if (dD != nullptr) dD[i - (int64_t)C * NP] = x;
    } else if (ddt_bias != nullptr) {
      ddt_bias[i - (int64_t)C * (NP + 1)] = x;
    }
  }
};

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
  const int ct = channel_tiles(a.C, a.G), np = 4 * NPL;
  const dim3 grid((unsigned)(ct * a.chunks), a.B);
  hipError_t e;
  if (a.chunks > 1) {
    hipLaunchKernelGGL((scan_fwd_kernel<T, NPL, true>), grid, dim3(kThreads), 0, s, a, ct);
    if ((e = noted(s)) != hipSuccess) return e;
    hipLaunchKernelGGL((scan_join_kernel<true>),
                       dim3((unsigned)(((int64_t)a.C * np + kThreads - 1) / kThreads), a.B),
                       dim3(kThreads), 0, s, a, np);
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
    hipLaunchKernelGGL((scan_join_kernel<false>),
                       dim3((unsigned)(((int64_t)a.C * np + kThreads - 1) / kThreads), a.B),
                       dim3(kThreads), 0, s, a, np);
    if ((e = noted(s)) != hipSuccess) return e;
  }
  hipLaunchKernelGGL((scan_bwd_kernel<T, NPL>), grid, dim3(kThreads), 0, s, a, ct);
  if ((e = noted(s)) != hipSuccess) return e;
  e = launch_column_sums(a.pA, (int64_t)a.B * a.chunks, (int64_t)a.C * (np + 2),
                         ScanSumStore{a.dA, a.dD, a.ddt_bias, a.C, a.N, np}, s);
  if (e != hipSuccess || a.T == 0) return e;
  const int64_t per = (int64_t)a.T * a.G * a.N;
  hipLaunchKernelGGL((scan_sum_bc<T>), dim3((unsigned)((per + kThreads - 1) / kThreads), a.B),
                     dim3(kThreads), 0, s, a, ct / a.G);
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
int scan_tile(int64_t N) { return N <= 16 ? 16 : (N <= 32 ? 8 : 4); }
int scan_channels() { return kChannels; }

int64_t scan_chunk(int64_t B, int64_t T, int64_t C, int64_t G, int64_t N, bool bwd) {
  const int64_t waves = B * channel_tiles(C, G) * kWaves;
  if (B == 0 || waves >= 2048 || T <= 64) return 0;
  int64_t parts = 4096 / waves;
  int64_t L = (T + parts - 1) / parts;
  L = (L + 15) / 16 * 16;
  if (L < 32) L = 32;
  return L < T ? L : 0;
}

hipError_t launch_scan_fwd(const ScanArgs& a, bool is_bf16, hipStream_t s) {
  return is_bf16 ? launch<bf16, false>(a, s) : launch<float, false>(a, s);
}
hipError_t launch_scan_bwd(const ScanArgs& a, bool is_bf16, hipStream_t s) {
  return is_bf16 ? launch<bf16, true>(a, s) : launch<float, true>(a, s);
}

}  // namespace gdr
