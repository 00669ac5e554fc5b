// Linear attention with a decay for each head on gfx950:
//   S_t = g_t S_{t-1} + v_t k_t^T,  y_t = scale S_t q_t,  g_t = exp(log_g_t).
// The adjoint D_t = scale dy_t q_t^T + g_{t+1} D_{t+1} gives dq = scale S^T dy,
// dk = D^T v, dv = D k: the forward's form with the roles of the tensors
// turned (and, for dk and dv, with time reversed), so one kernel serves all
// (gdr_lin.h):
//   state[o][i] <- g state + V[o] K[i];  out[o] = sum_i state[o][i] Q[i]
//   y: (Q, K, V) = (q, k, v);  dq: (dy, v, k);  dk: (v, dy, q);  dv: (k, q, dy).
// Where sequences times heads are too few for the device, sequences are cut
// into segments: one pass forms the segments' own ends (of k and v, or q and
// dy), a second joins them, and the main pass starts each segment from its
// state.  The forward's states around the segments are what it saves.
//
// dlog_g_t is what flows through the decay of step t: the sum of
//   A_ij = scale exp(..) (q_i k_j) (dy_i v_j) over i >= t > j,
// which is sum_{i >= t} (a_i - b_i) + <adjoint, state> behind the segment, with
// a_i the sum of A_ij over j < i (q_i times the part of dq_i that comes from
// earlier steps) and b_j that over i > j.  The term i = j, which both would
// hold, is left out of both, so that where all decays are strong no small
// difference of large sums is left.  It is left at a strong decay among weak
// ones: there dlog_g is off by units of the a_i and b_i behind it, as anywhere,
// but they are larger than itself.
#include "gdr_lin.h"

namespace gdr {
namespace {

constexpr int kThreads = 256;
// Steps up to which a forward call goes one step at a time.
constexpr int kFewSteps = 8;
constexpr int kStepRows = 4;  // of the state, of a group of lanes
// A log decay below which exp is 0 in fp32 (2^-150 rounds to 0): nothing flows
// through such a step.
constexpr float kNoFlow = -104.f;

// A step at a time.  LANES lanes own kStepRows rows of the state, each lane
// NV vectors of V neighbouring columns of every row, so that a row is read and
// written in whole cache lines.  Bound by the states, read and written once: 48
// requests of 32 heads of 128 x 128 (203 MB) take 34 us, 5.9 TB/s, over the same
// states again, 43 over others in turn (4.7).  (Lanes that own every 64th column,
// one element at a time: 54 and 61.)
template <typename T, int LANES, int NV, int V>
__global__ __launch_bounds__(kThreads) void lin_step_kernel(LinArgs a) {
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
  const int h = blockIdx.y, b = blockIdx.z, reps = a.Hv / a.Hk;
  const int o0 = (blockIdx.x * (kThreads / LANES) + group) * kStepRows;
  const Span sp = span_of(a.spans, b, a.T, a.rows);
  const int size = a.Dk * a.Dv;
  const int64_t whole = ((int64_t)b * a.Hv + h) * size;
  float S[kStepRows][NV][V];
#pragma unroll
  for (int j = 0; j < kStepRows; ++j)
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int o = o0 + j, i = (n * LANES + lane) * V;
      const bool in = a.S0 != nullptr && o < a.Dv && i < a.Dk;
      const Pack<float, V> x = in ? load_pack<float, V>(a.S0 + whole + o * a.Dk + i)
                                  : zero_pack<float, V>();
      unpack(x, S[j][n]);
    }
  auto store = [&](float* to) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < kStepRows; ++j)
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        const int o = o0 + j, i = (n * LANES + lane) * V;
        if (o < a.Dv && i < a.Dk) store_pack(to + o * a.Dk + i, S[j][n]);
      }
  };
  const int64_t slot = lin_slot(a, sp, b, 0);
  const bool save = a.ckpt != nullptr && sp.len > 0;
  if (save) store(a.ckpt + (slot * a.Hv + h) * size);
  for (int t = 0; t < sp.len; ++t) {
    const int64_t row = sp.first + t;
    const T* const Q = static_cast<const T*>(a.q) + row * a.q_stride + (int64_t)(h / reps) * a.Dk;
    const T* const K = static_cast<const T*>(a.k) + row * a.k_stride + (int64_t)(h / reps) * a.Dk;
    const T* const W = static_cast<const T*>(a.v) + row * a.v_stride + (int64_t)h * a.Dv;
    float q[NV][V], k[NV][V], v[kStepRows];
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int i = (n * LANES + lane) * V;
      const bool in = i < a.Dk;
      unpack(in ? load_pack<T, V>(Q + i) : zero_pack<T, V>(), q[n]);
      unpack(in ? load_pack<T, V>(K + i) : zero_pack<T, V>(), k[n]);
    }
#pragma unroll
    for (int j = 0; j < kStepRows; ++j) v[j] = o0 + j < a.Dv ? to_f32(W[o0 + j]) : 0.f;
    const float lg = lin_log_decay(a, row, h);
    const float g = expf(lg);
    if (lg > (float)kGrows) {  // (0 stays 0 where exp(lg) is past fp32's range)
#pragma unroll
      for (int j = 0; j < kStepRows; ++j)
#pragma unroll
        for (int n = 0; n < NV; ++n)
#pragma unroll
          for (int e = 0; e < V; ++e)
            S[j][n][e] = lg < __builtin_inff() ? lin_grow(S[j][n][e], lg) : __builtin_nanf("");
    } else {
#pragma unroll
      for (int j = 0; j < kStepRows; ++j)
#pragma unroll
        for (int n = 0; n < NV; ++n)
#pragma unroll
          for (int e = 0; e < V; ++e) S[j][n][e] *= g;
    }
    float x[kStepRows];
#pragma unroll
    for (int j = 0; j < kStepRows; ++j) {
      x[j] = 0.f;
#pragma unroll
      for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          S[j][n][e] = fmaf(v[j], k[n][e], S[j][n][e]);
          x[j] = fmaf(S[j][n][e], q[n][e], x[j]);
        }
      x[j] = rowsum16(x[j]);
      if constexpr (LANES >= 32) x[j] = swap16_sum(x[j], x[j]);
      if constexpr (LANES >= 64) x[j] = swap32_sum(x[j], x[j]);
    }
    if (lane == 0)
#pragma unroll
      for (int j = 0; j < kStepRows; ++j)
        if (o0 + j < a.Dv)
          st(static_cast<T*>(a.y), (row * a.Hv + h) * a.Dv + o0 + j, a.scale * x[j]);
  }
  if (a.S_T != nullptr) store(a.S_T + whole);
  if (save) store(a.ckpt + ((slot + 1) * a.Hv + h) * size);
}

// The states around the segments from their own ends, in place: forward slot
// s + 1 holds segment s's end, backward slot s holds segment s's adjoint at its
// begin and receives the one behind it.  Bound by the states' bytes, read and
// written: 2048 steps of 64 heads of 128 x 192 in 4 segments 11 us, 4.5 TB/s.
// (Each main pass joining what lies before its segment instead: no states
// between and no launch, but up to 64 loads a lane and segment where registers
// are short: training 494 us against 446, seven prompts 207 against 174.)
template <int V>
__global__ __launch_bounds__(kThreads) void lin_join_kernel(LinArgs a, int reverse) {
  const int h = blockIdx.y, b = blockIdx.z;
  const int size = a.Dk * a.Dv, at = (blockIdx.x * kThreads + threadIdx.x) * V;
  if (at >= size) return;
  const Span sp = span_of(a.spans, b, a.T, a.rows);
  const int n = (sp.len + a.seg - 1) / a.seg;
  const int64_t slot = lin_slot(a, sp, b, 0);
  const int64_t whole = ((int64_t)b * a.Hv + h) * size + at, step = (int64_t)a.Hv * size;
  float* const p = a.states + (slot * a.Hv + h) * size + at;
  const double* const d = a.decay + slot * a.Hv + h;
  const float* const first = reverse ? a.dS_T : a.S0;
  float S[V];
#pragma unroll
  for (int v = 0; v < V; ++v) S[v] = 0.f;
  if (first != nullptr) unpack(load_pack<float, V>(first + whole), S);
  float next[V];
  auto fetch = [&](int s) __attribute__((always_inline)) {
    unpack(load_pack<float, V>(p + (reverse ? n - 1 - s : s + 1) * step), next);
  };
  if (n > 0) fetch(0);
  for (int s = 0; s < n; ++s) {
    float x[V];
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = next[v];
    if (s + 1 < n) fetch(s + 1);
    const int m = reverse ? n - 1 - s : s;
    store_pack(p + m * step, S);
    const double log_g = d[(int64_t)m * a.Hv];
    const float g = lin_exp(log_g);
#pragma unroll
    for (int v = 0; v < V; ++v)
      S[v] = log_g > kGrows ? lin_grow(S[v], log_g) + x[v] : fmaf(g, S[v], x[v]);
  }
  if (!reverse && n > 0) store_pack(p + n * step, S);
  float* const last = reverse ? a.dS0 : a.S_T;
  if (last != nullptr) store_pack(last + whole, S);
}

// Sums of the fp32 parts over a key head's value heads, V columns a thread.
// Bound by the parts' bytes: 2048 rows of 64 x 192, twice (226 MB with the sums),
// 50 us, 4.5 TB/s.  (Heads of one key head in a workgroup, which would add them up
// in LDS: training 482 us against 451, shared by 64 heads 380 to 500 against 394,
// as too few workgroups are left.)
template <typename T, int V>
__global__ __launch_bounds__(kThreads) void lin_heads_sum(LinArgs a) {
  const int reps = a.Hv / a.Hk, b = blockIdx.y;
  const Span sp = span_of(a.spans, b, a.T, a.rows);
  const uint32_t units = a.Hk * a.Dk / V;  // of a row
  const int64_t n = (int64_t)sp.len * units;
  const float* const part = blockIdx.z == 0 ? a.dq_part : a.dk_part;
  T* const out = static_cast<T*>(blockIdx.z == 0 ? a.dq : a.dk);
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n;
       i += (int64_t)gridDim.x * kThreads) {
    const int64_t row = sp.first + i / units;
    const int c = (int)(i % units) * V, kh = c / a.Dk, d = c - kh * a.Dk;
    const float* const p = part + (row * a.Hv + kh * reps) * a.Dk + d;
    float s[V];
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = 0.f;
    int j = 0;
    for (; j + 4 <= reps; j += 4) {
      Pack<float, V> x[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) x[u] = load_pack<float, V>(p + (int64_t)(j + u) * a.Dk);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        float f[V];
        unpack(x[u], f);
#pragma unroll
        for (int v = 0; v < V; ++v) s[v] += f[v];
      }
    }
    for (; j < reps; ++j) {
      float f[V];
      unpack(load_pack<float, V>(p + (int64_t)j * a.Dk), f);
#pragma unroll
      for (int v = 0; v < V; ++v) s[v] += f[v];
    }
    store_pack(out + row * a.Hk * a.Dk + c, s);
  }
}

// Sum over a workgroup, in every thread.
__device__ __forceinline__ double block_sum(double x, double* red) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) x += __shfl_xor(x, m, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
  __syncthreads();
  return (red[0] + red[1]) + (red[2] + red[3]);
}

// dlog_g from the flows: a workgroup a segment and head walks the steps from
// the end, 256 at a time, sums in 64 bits.
__global__ __launch_bounds__(kThreads) void lin_flow_kernel(LinArgs a, int tiles) {
  __shared__ double red[kThreads / 64];
  const int sg = blockIdx.x, h = blockIdx.y, b = blockIdx.z, lane = threadIdx.x & 63,
            wave = threadIdx.x >> 6;
  const Span sp = span_of(a.spans, b, a.T, a.rows);
  const int begin = sg * a.seg;
  const int len = sp.len - begin < a.seg ? sp.len - begin : a.seg;
  if (len <= 0) {  // (the whole workgroup)
    if (a.per_head && threadIdx.x == 0)
      a.head_sums[((int64_t)b * a.segs + sg) * a.Hv + h] = 0.0;
    return;
  }
  const int64_t slot = lin_slot(a, sp, b, sg), n = (int64_t)a.Dk * a.Dv;
  const float* const S = a.ckpt + ((slot + 1) * a.Hv + h) * n;
  const float* const D = a.segs > 1          ? a.states + (slot * a.Hv + h) * n
                         : a.dS_T != nullptr ? a.dS_T + ((int64_t)b * a.Hv + h) * n
                                             : nullptr;
  double carry = 0.0, head = 0.0;
  if (D != nullptr) {
    // (16-byte loads where the states are whole vectors, four in flight)
    const int64_t whole = n % 4 == 0 ? n / 4 : 0;
    int64_t i = threadIdx.x;
    for (; i + 3 * kThreads < whole; i += 4 * kThreads) {
      float4 x[4], y[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        x[u] = reinterpret_cast<const float4*>(D)[i + u * kThreads];
        y[u] = reinterpret_cast<const float4*>(S)[i + u * kThreads];
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        carry += ((double)x[u].x * (double)y[u].x + (double)x[u].y * (double)y[u].y) +
                 ((double)x[u].z * (double)y[u].z + (double)x[u].w * (double)y[u].w);
    }
    for (i = whole > 0 ? 4 * (i - threadIdx.x) + threadIdx.x : threadIdx.x; i < n; i += kThreads)
      carry += (double)D[i] * (double)S[i];
    carry = block_sum(carry, red);
  }
  const float* const fa = a.flow + h * a.rows;
  const float* const fb = fa + (int64_t)tiles * a.rows * a.Hv;
  for (int t0 = (len - 1) & ~(kThreads - 1); t0 >= 0; t0 -= kThreads) {
    const int t = t0 + threadIdx.x;
    const int64_t row = sp.first + begin + t;
    double x = 0.0;
    if (t < len)
      for (int i = 0; i < tiles; ++i) {
        const int64_t at = (int64_t)i * a.rows * a.Hv + row;
        x += (double)fa[at] - (double)fb[at];
      }
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {  // sums over the wave's lanes from here on
      const double y = __shfl_down(x, m, 64);
      x += lane + m < 64 ? y : 0.0;
    }
    __syncthreads();
    if (lane == 0) red[wave] = x;
    __syncthreads();
    for (int w = wave + 1; w < kThreads / 64; ++w) x += red[w];
    x += carry;
    carry += (red[0] + red[1]) + (red[2] + red[3]);
    if (t < len) {
      if (lin_log_decay(a, row, h) < kNoFlow) x = 0.0;
      head += x;
      if (!a.per_head) {
        const int64_t at = row * a.Hv + h;
        if (a.g_bf16)
          st(static_cast<bf16*>(a.dlog_g), at, (float)x);
        else
          static_cast<float*>(a.dlog_g)[at] = (float)x;
      }
    }
  }
  if (!a.per_head) return;
  head = block_sum(head, red);
  if (threadIdx.x == 0) a.head_sums[((int64_t)b * a.segs + sg) * a.Hv + h] = head;
}

__global__ __launch_bounds__(kThreads) void lin_head_kernel(LinArgs a) {
  const int h = blockIdx.x * kThreads + threadIdx.x;
  if (h >= a.Hv) return;
  double s = 0.0;
  for (int64_t i = 0; i < (int64_t)a.B * a.segs; ++i) s += a.head_sums[i * a.Hv + h];
  st_weight(a.dlog_g, h, (float)s, a.g_bf16);
}

hipError_t noted(hipStream_t s) {
  const hipError_t e = hipGetLastError();
  note_launch(s);
  return e;
}

hipError_t join(const LinArgs& a, int reverse, hipStream_t s) {
  const int size = a.Dk * a.Dv, V = size % 4 == 0 ? 4 : 1;
  const dim3 grid((size / V + kThreads - 1) / kThreads, a.Hv, a.B);
  if (V == 4)
    hipLaunchKernelGGL(lin_join_kernel<4>, grid, dim3(kThreads), 0, s, a, reverse);
  else
    hipLaunchKernelGGL(lin_join_kernel<1>, grid, dim3(kThreads), 0, s, a, reverse);
  return noted(s);
}

hipError_t head_sums(const LinArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(lin_head_kernel, dim3((a.Hv + kThreads - 1) / kThreads), dim3(kThreads), 0, s,
                     a);
  return noted(s);
}

// Whether widths and strides let rows be read in whole vectors.
bool whole_vectors(const LinArgs& a, bool bf16) {
  const int64_t v = bf16 ? 8 : 4;
  return a.Dk % 8 == 0 && a.Dv % 8 == 0 && a.q_stride % v == 0 && a.k_stride % v == 0 &&
         a.v_stride % v == 0;
}

template <typename T>
hipError_t chunked(const LinArgs& a, const LinRole& r, int mode, hipStream_t s) {
  return r.vec ? lin_chunk<T, true>(a, r, mode, s) : lin_chunk<T, false>(a, r, mode, s);
}

template <typename T, int LANES, int NV, int V>
hipError_t step(const LinArgs& a, hipStream_t s) {
  constexpr int kRows = kThreads / LANES * kStepRows;
  hipLaunchKernelGGL((lin_step_kernel<T, LANES, NV, V>), dim3((a.Dv + kRows - 1) / kRows, a.Hv, a.B),
                     dim3(kThreads), 0, s, a);
  return noted(s);
}

template <typename T>
hipError_t fwd(const LinArgs& a, hipStream_t s) {
  if (a.T <= kFewSteps) {
    // (vectors of 16 bytes of the state, of 8 or 16 of the rows)
    const bool vec = a.Dk % 4 == 0 && a.q_stride % 4 == 0 && a.k_stride % 4 == 0;
    if (!vec) return step<T, 64, 4, 1>(a, s);
    return a.Dk <= 64 ? step<T, 16, 1, 4>(a, s)
                      : a.Dk <= 128 ? step<T, 32, 1, 4>(a, s) : step<T, 64, 1, 4>(a, s);
  }
  const int reps = a.Hv / a.Hk;
  LinRole r{};
  r.Q = a.q;
  r.K = a.k;
  r.V = a.v;
  r.sq = a.q_stride;
  r.sk = a.k_stride;
  r.sv = a.v_stride;
  r.dq = r.dk = reps;
  r.dv = 1;
  r.Ni = a.Dk;
  r.No = a.Dv;
  r.tiles = lin_tiles(r.Ni, r.No);
  r.ps = r.cs = a.scale;
  r.us = 1.f;
  r.vec = whole_vectors(a, sizeof(T) == 2);
  r.out = a.y;
  if (a.segs == 1) {
    r.first = a.S0;
    r.last = a.S_T;
    r.save = a.ckpt;
    return chunked<T>(a, r, kLinOut, s);
  }
  r.local = a.states;
  r.decay = a.decay;
  hipError_t e = chunked<T>(a, r, kLinState, s);
  if (e == hipSuccess) e = join(a, 0, s);
  r.first = a.states;
  r.slots = 1;
  return e == hipSuccess ? chunked<T>(a, r, kLinOut, s) : e;
}

template <typename T>
hipError_t bwd(const LinArgs& a, hipStream_t s) {
  const int reps = a.Hv / a.Hk;
  const int64_t wide = (int64_t)a.Hv * a.Dv;
  const int tiles = lin_tiles(a.Dv, a.Dk);
  const int mode = a.dlog_g != nullptr ? kLinFlow : kLinOut;
  hipError_t e = hipSuccess;
  if (a.B == 0) return head_sums(a, s);
  LinRole r{};
  r.vec = whole_vectors(a, sizeof(T) == 2);
  r.dq = 1;
  r.dk = 1;
  r.dv = r.dr = reps;
  // dq: (dy, v, k)
  r.Q = a.dy;
  r.K = a.v;
  r.V = a.k;
  r.R = a.q;
  r.sq = wide;
  r.sk = a.v_stride;
  r.sv = a.k_stride;
  r.sr = a.q_stride;
  r.Ni = a.Dv;
  r.No = a.Dk;
  r.tiles = tiles;
  r.ps = r.cs = a.scale;
  r.us = 1.f;
  r.transposed = 1;
  r.first = a.ckpt;
  r.slots = 1;
  r.out = reps > 1 ? nullptr : a.dq;
  r.part = a.dq_part;
  r.flow = a.flow;
  LinRole d = r;
  // dv: (k, q, dy)
  LinRole v = r;
  v.Q = a.k;
  v.K = a.q;
  v.V = a.dy;
  v.sq = a.k_stride;
  v.sk = a.q_stride;
  v.sv = wide;
  v.dq = v.dk = reps;
  v.dv = 1;
  v.Ni = a.Dk;
  v.No = a.Dv;
  v.tiles = lin_tiles(a.Dk, a.Dv);
  v.ps = v.us = a.scale;
  v.cs = 1.f;
  v.reverse = 1;
  v.transposed = 0;
  v.out = a.dv;
  v.part = nullptr;
  if (a.segs > 1) {
    v.first = nullptr;
    v.local = a.states;
    v.decay = a.decay;
    e = chunked<T>(a, v, kLinState, s);
    if (e == hipSuccess) e = join(a, 1, s);
    v.first = a.states;
  } else {
    v.first = a.dS_T;
    v.slots = 0;
    v.last = a.dS0;
  }
  // dk: (v, dy, q)
  d.Q = a.v;
  d.K = a.dy;
  d.V = a.q;
  d.R = a.k;
  d.sq = a.v_stride;
  d.sk = wide;
  d.sv = a.q_stride;
  d.sr = a.k_stride;
  d.ps = d.us = a.scale;
  d.cs = 1.f;
  d.reverse = 1;
  d.first = v.first;
  d.slots = v.slots;
  d.out = reps > 1 ? nullptr : a.dk;
  d.part = a.dk_part;
  d.flow = a.flow + (int64_t)tiles * a.rows * a.Hv;
  if (e == hipSuccess) {
    const LinRoles roles{{r, d, v}};
    e = r.vec ? lin_chunks<T, true>(a, roles, mode, s) : lin_chunks<T, false>(a, roles, mode, s);
  }
  if (e == hipSuccess && reps > 1) {
    const int V = a.Dk % 4 == 0 ? 4 : 1;
    const int64_t blocks = ((int64_t)a.T * a.Hk * a.Dk / V + kThreads - 1) / kThreads;
    const dim3 grid((unsigned)(blocks < 1 ? 1 : blocks > 2048 ? 2048 : blocks), a.B, 2);
    if (V == 4)
      hipLaunchKernelGGL((lin_heads_sum<T, 4>), grid, dim3(kThreads), 0, s, a);
    else
      hipLaunchKernelGGL((lin_heads_sum<T, 1>), grid, dim3(kThreads), 0, s, a);
    e = noted(s);
  }
  if (e == hipSuccess && mode == kLinFlow) {
    hipLaunchKernelGGL(lin_flow_kernel, dim3(a.segs, a.Hv, a.B), dim3(kThreads), 0, s, a, tiles);
    e = noted(s);
    if (e == hipSuccess && a.per_head) e = head_sums(a, s);
  }
  return e;
}

}  // namespace

// 128 columns a workgroup, which form P once for them, where the state leaves
// registers for two workgroups a compute unit (up to 128 contracted columns);
// 64 where it does not, and where 128 would leave a quarter of them empty.
// Measured when this was chosen, with operands of two pieces:
// training of 2048 steps, heads 16/64 of 192/128: 514 us; 128 columns for all
// widths 646, 64 only where 192 are contracted 520.  4 x 4096 steps of 32 heads
// of 128/128: 757 us, with 64 columns 903.
int lin_width(int64_t Ni, int64_t No) {
  return No <= 64 || Ni > 128 || (No > 128 && No <= 192) ? 64 : 128;
}
int lin_tiles(int64_t Ni, int64_t No) {
  const int w = lin_width(Ni, No);
  return (int)((No + w - 1) / w);
}

// Segments for 512 workgroups, two a compute unit, of 128 steps at least.  (256,
// 384, 768, 1024 and 1536 workgroups were all slower: fewer leave SIMDs with one
// wave, more repeat the state pass and wait for a second round.)
//
// Each sequence has a last segment that is cut off (of packed rows, half of one
// on average), so that a cut of all rows into 512 may leave a second round.  Where
// it does, that one of three cuts is taken whose steps are the fewest by this
// count: a round of workgroups takes its segment's steps and kLinEach more; more
// workgroups than one round take their share of all steps and half a segment;
// what is cut is walked again without outputs (0.45 of a pass) and joined (as 128
// steps).  Three draws each of 32 heads of 128/128: seven prompts in 6000 rows 159
// to 167 us, cut by rows alone 177 to 190; 20 of them (not cut) 108 to 120, by rows
// 213 to 219; 24 sequences in 16384 rows, 16 heads, training (not cut) 769 to 853,
// by rows 882 to 909, one round 1113 to 1142.  It loses 5% where it cuts to one
// round five sequences of 12000 rows, 16 heads of 64/64: 233, by rows 221.
constexpr double kLinEach = 96.0;
LinPlan lin_plan(int64_t B, int64_t T, int64_t rows, int64_t Hv, int64_t Dk, int64_t Dv) {
  LinPlan p{};
  const int64_t per = Hv * lin_tiles(Dk, Dv);  // workgroups of one cut through all rows
  const int64_t want = (512 + per - 1) / per;
  auto cut = [](int64_t steps, int64_t n) {
    const int64_t seg = ((steps + n - 1) / n + 63) / 64 * 64;
    return seg < 128 ? 128 : seg;
  };
  const bool dense = rows >= B * T;
  auto pieces = [&](int64_t seg) {
    return dense ? (double)(B * ((T + seg - 1) / seg)) : (double)rows / (double)seg + 0.5 * (double)B;
  };
  int64_t seg = cut(rows, want);
  if (T > seg && pieces(seg) > (double)want) {
    auto steps = [&](int64_t segment, double n) {
      const double x = (double)segment + kLinEach;
      return n <= (double)want ? x : ((double)rows + kLinEach * n) / (double)want + 0.5 * x;
    };
    auto split = [&](int64_t segment) { return 1.45 * steps(segment, pieces(segment)) + 128.0; };
    const int64_t one = dense ? cut(T, want > B ? want / B : 1)
                              : want > B / 2 ? cut(rows, want - B / 2) : seg;
    if (split(one) < split(seg)) seg = one;
    if (steps(T, (double)B) < split(seg)) seg = T;
  }
  if (T <= seg) seg = rows < T ? (T < 1 ? 1 : T) : (rows < 1 ? 1 : rows);  // one
  p.seg = seg;
  p.segs = T > seg ? (T + seg - 1) / seg : 1;
  p.slots = rows / seg + 2 * B + 1;
  return p;
}

hipError_t launch_lin_fwd(const LinArgs& a, bool is_bf16, hipStream_t s) {
  return is_bf16 ? fwd<bf16>(a, s) : fwd<float>(a, s);
}
hipError_t launch_lin_bwd(const LinArgs& a, bool is_bf16, hipStream_t s) {
  return is_bf16 ? bwd<bf16>(a, s) : bwd<float>(a, s);
}

}  // namespace gdr
