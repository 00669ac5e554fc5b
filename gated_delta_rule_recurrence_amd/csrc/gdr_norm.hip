// Group norm over channels-last rows on gfx950.  A group is D = C / G
// neighbouring channels of one row:
//   xh = (x - mu) r,  r = 1 / sqrt(mean((x - mu)^2) + eps)   (mu = 0: RMS)
//   n = xh w + b;  y = act(n), or n act(z) with a gate z.
// Backward, with mu and r from the forward:
//   dn = dy act(z) (dy act'(n) without a gate),  dz = dy n act'(z),
//   e = dn w,  dx = r (e - mean(e) - xh mean(e xh))   (mean(e): centred only)
//   dw = sum over rows dn xh,  db = sum over rows dn.
// Bound by HBM bytes: every tensor once.  Measured (bf16, groups of 128 with
// a gate; a large copy reaches 4.98 TB/s): forward over 2048 x 8192 20 us, 5.1
// TB/s; over 8192 x 8192 75 us, 5.4 TB/s; backward over those 125 us, 5.4 TB/s.
//
// Mapping: LANES lanes own one group, each NV vectors of V channels, kept in
// registers between the statistics and the output.  Groups of up to 64
// vectors share a wave (LANES = 8 .. 64), wider ones take a whole workgroup.
// A "slab" is what one wave (one workgroup, for LANES > 64) takes at a time:
// consecutive groups of the flattened [rows * G] list.  A wave walks the list
// in steps of a multiple of `period` groups, itself a multiple of G, so that
// a lane meets the same channels all the way: it holds their weights, and the
// backward its sums dw and db, in registers.
#include "gdr_layer.h"

namespace gdr {
namespace {

constexpr int kThreads = 256;

// Sum over the LANES lanes of a group, the same bits in every lane.
template <int LANES>
__device__ __forceinline__ float group_sum(float x, float* red) {
  x += dpp<kDppQuadSwap1>(x);
  x += dpp<kDppQuadSwap2>(x);
  x += dpp<kDppHalfMirror>(x);
  if constexpr (LANES >= 16) x += dpp<kDppMirror>(x);
  if constexpr (LANES >= 32) x = swap16_sum(x, x);
  if constexpr (LANES >= 64) x = swap32_sum(x, x);
  if constexpr (LANES > 64) {
    __syncthreads();  // the last sum has been read
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
    __syncthreads();
    x = red[0];
#pragma unroll
    for (int i = 1; i < LANES / 64; ++i) x += red[i];
  }
  return x;
}

template <typename T, int LANES, int NV, int V>
struct Norm {
  static constexpr int kBlock = LANES > 64 ? LANES : kThreads;
  static constexpr int kUnits = LANES > 64 ? 1 : 64 / LANES;  // groups of one slab
  static constexpr int kSlabs = LANES > 64 ? 1 : kThreads / 64;  // slabs of a workgroup at once

  // channel of vector i of this lane inside its group
  static __device__ __forceinline__ int at(int lane, int i) { return (i * LANES + lane) * V; }

  static __device__ __forceinline__ void weights(const NormArgs& a, int lane, int g,
                                                 float (&w)[NV][V], float (&b)[NV][V]) {
    const int64_t base = a.shared ? 0 : (int64_t)g * a.D, count = a.shared ? a.D : a.C;
    Weights<V, (V > 1)> wr[NV], br[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      // (a group is whole vectors)
      const int64_t first = at(lane, i) < a.D ? base + at(lane, i) : count;
      wr[i].load(a.w, first, count, a.w_bf16);
      br[i].load(a.bias, first, count, a.w_bf16);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      wr[i].get(a.w_bf16, w[i]);
      br[i].get(a.w_bf16, b[i]);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const bool in = at(lane, i) + v < a.D;
        w[i][v] = in ? (a.w != nullptr ? w[i][v] : 1.f) : 0.f;
        b[i][v] = in ? b[i][v] : 0.f;
      }
    }
  }
  // A group's channels of one tensor (zeros past the group's end).
  static __device__ __forceinline__ void load(const void* p, int64_t off, int lane, int D, bool ok,
                                              Pack<T, V> (&x)[NV]) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      x[i] = ok && at(lane, i) < D ? load_pack<T, V>(static_cast<const T*>(p) + off + at(lane, i))
                                   : zero_pack<T, V>();
  }
};

// Where a lane walks: its channels' group g, its first row and the rows from
// one turn to the next (rows G fits in 31 bits).
struct Walk {
  int g;
  int64_t row, step;
};
template <typename P>
__device__ __forceinline__ Walk walk_of(const NormArgs& a, int period, int slabs, int part,
                                        int parts, int wave, int sub) {
  const int slab = (int)blockIdx.x % slabs;
  const int place = slab * P::kUnits + sub;
  const int turns = period / a.G;  // rows of a period
  return Walk{place % a.G, (int64_t)(part * P::kSlabs + wave) * turns + place / a.G,
              (int64_t)parts * P::kSlabs * turns};
}

template <typename T, int LANES, int NV, int V>
__global__ __launch_bounds__((Norm<T, LANES, NV, V>::kBlock)) void norm_fwd_kernel(NormArgs a,
                                                                                   int period,
                                                                                   int slabs) {
  using P = Norm<T, LANES, NV, V>;
  __shared__ float red[LANES > 64 ? LANES / 64 : 1];
  const int lane = LANES > 64 ? threadIdx.x : threadIdx.x & (LANES - 1);
  const int wave = LANES > 64 ? 0 : threadIdx.x >> 6;
  const int sub = LANES > 64 ? 0 : (threadIdx.x & 63) / LANES;
  const Walk k = walk_of<P>(a, period, slabs, blockIdx.x / slabs, gridDim.x / slabs, wave, sub);
  const int64_t go = (int64_t)k.g * a.D;
  Pack<T, V> xn[NV], zn[NV];  // the next turn's rows
  auto fetch = [&](int64_t row) __attribute__((always_inline)) {
    P::load(a.x, row * a.x_stride + go, lane, a.D, row < a.rows, xn);
    if (a.z != nullptr) P::load(a.z, row * a.z_stride + go, lane, a.D, row < a.rows, zn);
  };
  fetch(k.row);
  float w[NV][V], bias[NV][V];
  P::weights(a, lane, k.g, w, bias);
  const float inv = 1.f / (float)a.D;
  for (int64_t row = k.row; row < a.rows; row += k.step) {
    Pack<T, V> xr[NV], zr[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      xr[i] = xn[i];
      zr[i] = zn[i];
    }
    fetch(row + k.step);
    float x[NV][V], mu = 0.f, s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) unpack(xr[i], x[i]);
    if (a.center) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) s += x[i][v];
      mu = group_sum<LANES>(s, red) * inv;
      s = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) x[i][v] = P::at(lane, i) + v < a.D ? x[i][v] - mu : 0.f;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) s = fmaf(x[i][v], x[i][v], s);
    const float r = 1.f / sqrtf(fmaf(group_sum<LANES>(s, red), inv, a.eps));
    if (a.stats != nullptr && lane == 0) {
      a.stats[2 * (row * a.G + k.g)] = mu;
      a.stats[2 * (row * a.G + k.g) + 1] = r;
    }
    T* const y = static_cast<T*>(a.y) + row * a.C + go;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float o[V], z[V];
      if (a.z != nullptr) unpack(zr[i], z);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float n = fmaf(x[i][v] * r, w[i][v], bias[i][v]);
        const float in = a.z != nullptr ? z[v] : n;
        o[v] = a.act ? silu(in) : in;
        if (a.z != nullptr) o[v] *= n;
      }
      if (P::at(lane, i) < a.D) store_pack(y + P::at(lane, i), o);
    }
  }
}

template <typename T, int LANES, int NV, int V>
__global__ __launch_bounds__((Norm<T, LANES, NV, V>::kBlock)) void norm_bwd_kernel(
    NormArgs a, int period, int slabs) {
  using P = Norm<T, LANES, NV, V>;
  __shared__ float red[LANES > 64 ? LANES / 64 : 1];
  const int lane = LANES > 64 ? threadIdx.x : threadIdx.x & (LANES - 1);
  const int wave = LANES > 64 ? 0 : threadIdx.x >> 6;
  const int sub = LANES > 64 ? 0 : (threadIdx.x & 63) / LANES;
  const int part = blockIdx.x / slabs;
  const Walk k = walk_of<P>(a, period, slabs, part, gridDim.x / slabs, wave, sub);
  const int64_t go = (int64_t)k.g * a.D;
  float w[NV][V], bias[NV][V], dw[NV][V], db[NV][V];
  P::weights(a, lane, k.g, w, bias);
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int v = 0; v < V; ++v) dw[i][v] = db[i][v] = 0.f;
  const float inv = 1.f / (float)a.D;

  for (int64_t row = k.row; row < a.rows; row += k.step) {
    Pack<T, V> xr[NV], zr[NV], dyr[NV];
    P::load(a.x, row * a.x_stride + go, lane, a.D, true, xr);
    P::load(a.dy, row * a.C + go, lane, a.D, true, dyr);
    if (a.z != nullptr) P::load(a.z, row * a.z_stride + go, lane, a.D, true, zr);
    const float mu = a.stats[2 * (row * a.G + k.g)], r = a.stats[2 * (row * a.G + k.g) + 1];
    float xh[NV][V], e[NV][V], se = 0.f, sx = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float dz[V], z[V], dy[V];
      unpack(xr[i], xh[i]);
      unpack(dyr[i], dy);
      if (a.z != nullptr) unpack(zr[i], z);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const bool in = P::at(lane, i) + v < a.D;
        xh[i][v] = in ? (xh[i][v] - mu) * r : 0.f;
        const float n = fmaf(xh[i][v], w[i][v], bias[i][v]);
        float dn = dy[v];
        if (a.z != nullptr) {
          const float sg = a.act ? sigmoid(z[v]) : 1.f;
          dz[v] = a.act ? dy[v] * n * dsilu(z[v], sg) : dy[v] * n;
          dn *= z[v] * sg;
        } else if (a.act) {
          dn *= dsilu(n, sigmoid(n));
        }
        dn = in ? dn : 0.f;
        dw[i][v] = fmaf(dn, xh[i][v], dw[i][v]);
        db[i][v] += dn;
        e[i][v] = dn * w[i][v];
        se += e[i][v];
        sx = fmaf(e[i][v], xh[i][v], sx);
      }
      if (a.z != nullptr && P::at(lane, i) < a.D)
        store_pack(static_cast<T*>(a.dz) + row * a.C + go + P::at(lane, i), dz);
    }
    sx = group_sum<LANES>(sx, red) * inv;
    se = a.center ? group_sum<LANES>(se, red) * inv : 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float o[V];
#pragma unroll
      for (int v = 0; v < V; ++v) o[v] = r * (e[i][v] - se - xh[i][v] * sx);
      if (P::at(lane, i) < a.D)
        store_pack(static_cast<T*>(a.dx) + row * a.C + go + P::at(lane, i), o);
    }
  }
  if (a.dw == nullptr && a.dbias == nullptr) return;
  // Sums over the workgroup's waves (and, for a shared weight, over a wave's
  // groups), then part[part][2][period][D], or part[workgroup][2][D] shared.
  const int64_t width = a.shared ? a.D : (int64_t)period * a.D;
  const int64_t place = (int64_t)((int)blockIdx.x % slabs) * P::kUnits + sub;
  float* const p = a.part + (a.shared ? (int64_t)blockIdx.x * 2 * width
                                      : part * 2 * width + place * a.D);
  __shared__ float sum[LANES > 64 ? 1 : P::kSlabs - 1][2][64];
  const int wl = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float s0 = dw[i][v], s1 = db[i][v];
      const int d = P::at(lane, i) + v;
      if constexpr (LANES <= 64) {
        if (a.shared)
#pragma unroll
          for (int m = LANES; m < 64; m <<= 1) {
            s0 += __shfl_xor(s0, m, 64);
            s1 += __shfl_xor(s1, m, 64);
          }
        __syncthreads();
        if (wave > 0) {
          sum[wave - 1][0][wl] = s0;
          sum[wave - 1][1][wl] = s1;
        }
        __syncthreads();
        if (wave == 0)
#pragma unroll
          for (int q = 0; q < P::kSlabs - 1; ++q) {
            s0 += sum[q][0][wl];
            s1 += sum[q][1][wl];
          }
      }
      if (wave == 0 && d < a.D && (!a.shared || sub == 0)) {
        p[d] = s0;
        p[width + d] = s1;
      }
    }
}

// Column c of a partial row [2][reps][W]: the repeats of W (a period that
// holds the weight's channels more than once) are further rows.
struct NormSumStore {
  void* dw;
  void* dbias;
  int64_t W;
  int w_bf16;
  __device__ void operator()(int64_t c, float x) const {
    if (c < W) {
      if (dw != nullptr) st_weight(dw, c, x, w_bf16);
    } else if (dbias != nullptr) {
      st_weight(dbias, c - W, x, w_bf16);
    }
  }
};

// Sums of part[parts][2][reps][W] to [2][W]: 16 columns and 64 row lanes over
// parts x reps, the row lanes' sums then added in order.
constexpr int kSumRows = 64;
__global__ __launch_bounds__(kSumCols* kSumRows) void norm_sums(const float* __restrict__ part,
                                                                int parts, int reps,
                                                                NormSumStore store) {
  __shared__ float red[kSumRows][kSumCols + 1];
  const int tc = threadIdx.x % kSumCols, tr = threadIdx.x / kSumCols;
  const int64_t c = (int64_t)blockIdx.x * kSumCols + tc;
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  if (c < 2 * store.W) {
    const int64_t half = c / store.W, d = c % store.W, block = 2 * reps * store.W;
    for (int k = 0; k < reps; ++k) {
      const float* const p = part + (half * reps + k) * store.W + d;
      int r = tr;
      for (; r + 3 * kSumRows < parts; r += 4 * kSumRows)
#pragma unroll
        for (int u = 0; u < 4; ++u) s[u] += p[(r + u * kSumRows) * block];
      for (; r < parts; r += kSumRows) s[0] += p[r * block];
    }
  }
  red[tr][tc] = (s[0] + s[1]) + (s[2] + s[3]);
  __syncthreads();
  if (tr < 4) {  // four partial chains, then their sum
    float t = red[tr][tc];
#pragma unroll
    for (int k = 1; k < kSumRows / 4; ++k) t += red[tr + 4 * k][tc];
    red[tr][tc] = t;
  }
  __syncthreads();
  if (tr == 0 && c < 2 * store.W)
    store(c, (red[0][tc] + red[1][tc]) + (red[2][tc] + red[3][tc]));
}

template <typename T, int LANES, int NV, int V>
hipError_t fwd(const NormArgs& a, const NormPlan& p, hipStream_t s) {
  using P = Norm<T, LANES, NV, V>;
  hipLaunchKernelGGL((norm_fwd_kernel<T, LANES, NV, V>), dim3((unsigned)(p.slabs * p.parts)),
                     dim3(P::kBlock), 0, s, a, (int)p.period, (int)p.slabs);
  const hipError_t e = hipGetLastError();
  note_launch(s);
  return e;
}

template <typename T, int LANES, int NV, int V>
hipError_t bwd(const NormArgs& a, const NormPlan& p, hipStream_t s) {
  using P = Norm<T, LANES, NV, V>;
  hipLaunchKernelGGL((norm_bwd_kernel<T, LANES, NV, V>), dim3((unsigned)(p.slabs * p.parts)),
                     dim3(P::kBlock), 0, s, a, (int)p.period, (int)p.slabs);
  hipError_t e = hipGetLastError();
  note_launch(s);
  if (e != hipSuccess || (a.dw == nullptr && a.dbias == nullptr)) return e;
  const int64_t W = a.shared ? a.D : a.C;
  const int64_t parts = a.shared ? p.parts * p.slabs : p.parts;
  const int64_t reps = a.shared ? 1 : p.period / a.G;
  hipLaunchKernelGGL(norm_sums, dim3((unsigned)((2 * W + kSumCols - 1) / kSumCols)),
                     dim3(kSumCols * kSumRows), 0, s, a.part, (int)parts, (int)reps,
                     NormSumStore{a.dw, a.dbias, W, a.w_bf16});
  e = hipGetLastError();
  note_launch(s);
  return e;
}

template <typename T, bool BWD, int LANES, int NV, int V>
hipError_t go(const NormArgs& a, const NormPlan& p, hipStream_t s) {
  return BWD ? bwd<T, LANES, NV, V>(a, p, s) : fwd<T, LANES, NV, V>(a, p, s);
}

template <typename T, bool BWD, int NV, int V>
hipError_t launch_lanes(const NormArgs& a, const NormPlan& p, hipStream_t s) {
  if constexpr (NV == 1) {
    if (p.lanes == 8) return go<T, BWD, 8, 1, V>(a, p, s);
    if (p.lanes == 16) return go<T, BWD, 16, 1, V>(a, p, s);
    if (p.lanes == 32) return go<T, BWD, 32, 1, V>(a, p, s);
  }
  if (p.lanes == 64) return go<T, BWD, 64, NV, V>(a, p, s);
  if constexpr (NV * V >= 8)
    if (p.lanes == 256) return go<T, BWD, 256, NV, V>(a, p, s);
  if constexpr (NV * V == 16)
    if (p.lanes == 512) return go<T, BWD, 512, NV, V>(a, p, s);
  return hipErrorInvalidValue;
}

template <typename T, bool BWD, int V>
hipError_t launch_v(const NormArgs& a, const NormPlan& p, hipStream_t s) {
  switch (p.nv) {
    case 1: return launch_lanes<T, BWD, 1, V>(a, p, s);
    case 2: return launch_lanes<T, BWD, 2, V>(a, p, s);
    case 4:
      if constexpr (V <= 4) return launch_lanes<T, BWD, 4, V>(a, p, s);
      break;
    case 16:
      if constexpr (V == 1) return launch_lanes<T, BWD, 16, V>(a, p, s);
      break;
  }
  return hipErrorInvalidValue;
}

template <typename T, bool BWD>
hipError_t launch(const NormArgs& a, const NormPlan& p, hipStream_t s) {
  return p.vec ? launch_v<T, BWD, 16 / sizeof(T)>(a, p, s) : launch_v<T, BWD, 1>(a, p, s);
}

int64_t gcd64(int64_t a, int64_t b) { return b == 0 ? a : gcd64(b, a % b); }

}  // namespace

// Lanes and vectors of a group: at most 16 channels per lane (the backward
// holds six values per channel), so groups of up to 1024 channels take (part
// of) a wave and up to 8192 a workgroup.
bool norm_plan(int64_t rows, int64_t C, int64_t G, int64_t xs, int64_t zs, bool bf16, NormPlan* p) {
  const int64_t D = C / G, V = bf16 ? 8 : 4;
  p->vec = D % V == 0 && xs % V == 0 && zs % V == 0;
  const int64_t v = p->vec ? V : 1, n = (D + v - 1) / v;  // vectors of a group
  const int most_nv = (int)(16 / v);
  if (n <= 64) {
    p->lanes = 8;
    while (p->lanes < n) p->lanes *= 2;
  } else if (n <= 64 * most_nv) {
    p->lanes = 64;
  } else {
    p->lanes = 256;
    while (p->lanes * most_nv < n) p->lanes *= 2;
    if (p->lanes > 512) return false;
  }
  p->nv = 1;
  while (p->lanes * p->nv < n) p->nv *= 2;
  if (p->nv == 8 || (p->nv < most_nv && p->lanes > 256)) p->nv = most_nv;
  const int64_t per = p->lanes > 64 ? 1 : 64 / p->lanes;
  p->period = G / gcd64(G, per) * per;
  p->slabs = p->period / per;
  // Workgroups in all: three per compute unit of 256 (at 512, 768, 1024, 2048
  // the training step of 131072 x 2048 in groups of 128 takes 81 + 144 + 5,
  // 76 + 125 + 5, 79 + 130 + 5, 82 + 131 + 8 us; 1237 rows of six groups of 185
  // in fp32 7 + 9 + 3, 7 + 9 + 4, 8 + 10 + 4, 9 + 11 + 4: more leave a wave
  // too few rows for its weights).  Where a workgroup walks as one, 131072
  // threads (4096 x 8192, 512 lanes: 48 + 85 + 8 at 256, 46 + 102 + 12 at 512;
  // 16384 x 4096, 256 lanes: 86 + 181 + 5 at 256, 75 + 131 + 7 at 512, 70 + 151
  // + 11 at 1024).  And no more than there are units for.
  const int64_t walkers = p->lanes > 64 ? 1 : kThreads / 64;
  const int64_t want = p->lanes > 64 ? 131072 / p->lanes : 768;
  const int64_t turns = (rows * G + p->period - 1) / p->period;
  int64_t parts = (want + p->slabs - 1) / p->slabs;
  const int64_t most = (turns + walkers - 1) / walkers;
  if (parts > most) parts = most;
  p->parts = parts < 1 ? 1 : parts;
  return true;
}

hipError_t launch_norm_fwd(const NormArgs& a, const NormPlan& p, bool is_bf16, hipStream_t s) {
  return is_bf16 ? launch<bf16, false>(a, p, s) : launch<float, false>(a, p, s);
}
hipError_t launch_norm_bwd(const NormArgs& a, const NormPlan& p, bool is_bf16, hipStream_t s) {
  return is_bf16 ? launch<bf16, true>(a, p, s) : launch<float, true>(a, p, s);
}

}  // namespace gdr
