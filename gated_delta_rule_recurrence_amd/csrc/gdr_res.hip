// The norms before and after a block with its gate and residual sum, on
// gfx950.  Per row, N(a; w, b) = (a - mu) r (w + offset) + b with
// r = 1 / sqrt(mean((a - mu)^2) + eps) (mu = 0: a root mean square norm):
//   n = N(x; post), or x;  h = residual + alpha gate n;  y = N(h; pre).
// Backward, with both norms' mu and r from the forward and h formed again
// (in fp32, as the forward had it, so h need not be kept):
//   e = dy (w + offset),  dh' = dh + r (e - mean(e) - hh mean(e hh)),  dr = dh'
//   dgate = alpha dh' n,  dn = alpha gate dh',  dx from dn as dh' from dy.
// Bound by HBM bytes: every tensor once.  8192 x 4096 in bf16: forward 47 to 51 us
// (268 MB, 5.2 to 5.7 TB/s, part of it from the memory-side cache), backward 94 to
// 97 (403 MB, 4.2 TB/s, its vector units half busy), the sums over rows 6; 6000 x
// 5120 with an fp32 residual, forward 71 to 76 us (369 MB, 4.9 to 5.2 TB/s).
//
// Mapping: LANES lanes own one row, each NV vectors of V channels, in registers
// from the loads to the stores; rows of up to 64 vectors take a wave, wider ones
// a workgroup.  A workgroup walks neighbouring rows, which lie inside one row
// of the gate or are whole gate rows, so that it holds weights, gate and the
// backward's sums over rows in registers.
#include "gdr_layer.h"

namespace gdr {
namespace {

constexpr int kThreads = 256;

// Waves of a row.
template <int LANES>
constexpr int kRowWaves = LANES > 64 ? LANES / 64 : 1;

// Sums of two values over the LANES lanes of a row, the same bits in every
// lane.  Every call of a kernel takes the other of two buffers than the call
// before it, which `turn` counts (a row may make a single call, always from the
// same place), so one barrier does for each: a wave that writes a buffer again
// has passed the barrier of the call between, behind every wave's reads of it.
template <int LANES>
__device__ __forceinline__ void row_sums(float& x, float& y,
                                         float (*buffers)[kRowWaves<LANES>][2], int& turn) {
  x = rowsum16(x);
  y = rowsum16(y);
  x = swap16_sum(x, x);
  y = swap16_sum(y, y);
  x = swap32_sum(x, x);
  y = swap32_sum(y, y);
  if constexpr (LANES > 64) {
    float (*const red)[2] = buffers[turn];
    turn ^= 1;
    if ((threadIdx.x & 63) == 0) {
      red[threadIdx.x >> 6][0] = x;
      red[threadIdx.x >> 6][1] = y;
    }
    lds_barrier();
    x = red[0][0];
    y = red[0][1];
#pragma unroll
    for (int i = 1; i < LANES / 64; ++i) {
      x += red[i][0];
      y += red[i][1];
    }
  }
}

// Whether the next row's loads fly while this one is worked on: not where the
// registers do not hold it (1024 lanes have 128 each; single elements take one
// each): 6000 x 5120 forward 91 us with, 68 without; 1237 x 1110 backward in
// fp32 47 and 21.  8192 x 4096 backward, with the kernel as it was then, 160 us
// without and 114 with.
template <int LANES, int V>
constexpr bool kAhead = LANES < 1024 && V > 1;

template <int LANES>
struct Res {
  static constexpr int kBlock = LANES > 64 ? LANES : kThreads;
  static constexpr int kWalkers = LANES > 64 ? 1 : kThreads / 64;  // rows at a time
};

// N consecutive channels of a parameter, or `other` where it is absent.
template <int V>
__device__ __forceinline__ void parameter(const void* p, int c, int C, int is_bf16, float offset,
                                          float other, float (&w)[V]) {
  Weights<V, (V > 1)> raw;
  raw.load(p, c, C, is_bf16);
  raw.get(is_bf16, w);
#pragma unroll
  for (int v = 0; v < V; ++v) w[v] = p != nullptr ? w[v] + offset : other;
}

// A row's C elements as a buffer (zeros past its end), of no bytes where the
// row or the tensor is not there.
template <typename R>
__device__ __forceinline__ Buffer row_of(const void* p, int64_t row, int64_t stride, int C,
                                         bool there) {
  return buffer_of(p, there ? row * stride * (int64_t)sizeof(R) : 0,
                   there ? C * (int64_t)sizeof(R) : 0);
}

// V neighbouring elements as loaded: of bf16 a vector of up to 16 bytes, of
// floats one or two.
template <typename R, int V>
struct Raw {
  static constexpr int VR = V * (int)sizeof(R) <= 16 ? V : 16 / (int)sizeof(R);
  Pack<R, VR> p[V / VR];
  __device__ __forceinline__ void load(Buffer row, int c) {
#pragma unroll
    for (int k = 0; k < V / VR; ++k) p[k] = get_pack<R, VR>(row, (c + k * VR) * sizeof(R));
  }
  __device__ __forceinline__ void get(float (&f)[V]) const {
#pragma unroll
    for (int k = 0; k < V / VR; ++k) {
      float g[VR];
      unpack(p[k], g);
#pragma unroll
      for (int v = 0; v < VR; ++v) f[k * VR + v] = g[v];
    }
  }
};
// A gate's, of either type.
template <int V>
struct RawGate {
  Raw<bf16, V> lo;
  Raw<float, V> hi;
  __device__ __forceinline__ void load(const ResArgs& a, int64_t row, int c) {
    if (a.gate_bf16)
      lo.load(row_of<bf16>(a.gate, row, a.gate_stride, a.C, true), c);
    else
      hi.load(row_of<float>(a.gate, row, a.gate_stride, a.C, true), c);
  }
  __device__ __forceinline__ void get(const ResArgs& a, float (&f)[V]) const {
    if (a.gate_bf16)
      lo.get(f);
    else
      hi.get(f);
  }
};
template <typename R, int V>
__device__ __forceinline__ void put_stream(void* p, int64_t off, const float (&f)[V]) {
  constexpr int VR = V == 1 ? 1 : (V * (int)sizeof(R) <= 16 ? V : 16 / (int)sizeof(R));
#pragma unroll
  for (int k = 0; k < V / VR; ++k) {
    float g[VR];
#pragma unroll
    for (int v = 0; v < VR; ++v) g[v] = f[k * VR + v];
    store_pack(static_cast<R*>(p) + off + k * VR, g);
  }
}

// Rows of a workgroup: [first, last) of the gate rows [gate, gate_end).
struct Walk {
  int64_t first, last;
};
__device__ __forceinline__ Walk walk_of(const ResArgs& a, const ResPlan& p) {
  const int64_t per = a.gate_rows > 1 ? a.gate_rows : a.rows;  // of one gate row
  int64_t first, last;
  if (p.per_gate > 1) {
    const int64_t g = blockIdx.x / p.per_gate;
    first = g * per + blockIdx.x % p.per_gate * p.step;
    last = first + p.step;
    last = last < (g + 1) * per ? last : (g + 1) * per;
  } else {
    first = blockIdx.x * p.step;
    last = first + p.step;
  }
  return Walk{first, last < a.rows ? last : a.rows};
}

template <typename T, typename R, int LANES, int NV, int V>
__global__ __launch_bounds__((Res<LANES>::kBlock)) void res_fwd_kernel(ResArgs a,
                                                                               ResPlan p) {
  using P = Res<LANES>;
  __shared__ float red[2][kRowWaves<LANES>][2];
  const int lane = threadIdx.x % LANES, wave = LANES > 64 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Walk k = walk_of(a, p);
  const float inv = 1.f / (float)a.C;
  int turn = 0;  // of row_sums
  Raw<T, V> xn[NV];  // the next row
  Raw<R, V> rn[NV];
  RawGate<V> gn[NV];
  const bool row_gate = a.gate != nullptr && a.gate_rows == 1;
  auto fetch = [&](int64_t row) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * LANES + lane) * V;
      const bool there = row < k.last;
      xn[i].load(row_of<T>(a.x, row, a.x_stride, a.C, there), c);
      rn[i].load(row_of<R>(a.r, row, a.r_stride, a.C, there), c);
      if (row_gate && there) gn[i].load(a, row, c);
    }
  };
  if constexpr (kAhead<LANES, V>) fetch(k.first + wave);
  float pw[NV][V], pb[NV][V], w[NV][V], wb[NV][V], gate[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * LANES + lane) * V, at = c < a.C ? c : a.C;
    parameter(a.post_w, at, a.C, a.w_bf16, a.offset, 1.f, pw[i]);
    parameter(a.post_b, at, a.C, a.w_bf16, 0.f, 0.f, pb[i]);
    parameter(a.pre_w, at, a.C, a.w_bf16, a.offset, 1.f, w[i]);
    parameter(a.pre_b, at, a.C, a.w_bf16, 0.f, 0.f, wb[i]);
#pragma unroll
    for (int v = 0; v < V; ++v) gate[i][v] = 1.f;
  }
  int64_t held = -1;  // the gate's row in registers
  for (int64_t row = k.first + wave; row < k.last; row += P::kWalkers) {
    float x[NV][V], h[NV][V], s = 0.f, mu = 0.f, zero = 0.f;
    const int64_t g = row / a.gate_rows;
    if (a.gate != nullptr && !row_gate && g != held) {
      held = g;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * LANES + lane) * V;
        RawGate<V> raw;
        raw.load(a, g, c);
        raw.get(a, gate[i]);
      }
    }
    if constexpr (!kAhead<LANES, V>) fetch(row);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      xn[i].get(x[i]);
      rn[i].get(h[i]);
      if (row_gate) gn[i].get(a, gate[i]);
    }
    if constexpr (kAhead<LANES, V>) fetch(row + P::kWalkers);
    float mu1 = 0.f, r1 = 0.f, r2 = 0.f;
    if (a.post) {
      if (a.center) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int v = 0; v < V; ++v) s += x[i][v];
        row_sums<LANES>(s, zero, red, turn);
        mu1 = s * inv;
      }
      s = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          x[i][v] = (i * LANES + lane) * V < a.C ? x[i][v] - mu1 : 0.f;
          s = fmaf(x[i][v], x[i][v], s);
        }
      row_sums<LANES>(s, zero, red, turn);
      r1 = 1.f / sqrtf(fmaf(s, inv, a.eps));
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) x[i][v] = fmaf(x[i][v] * r1, pw[i][v], pb[i][v]);
    }
    s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * LANES + lane) * V;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        h[i][v] = fmaf(a.alpha * gate[i][v], x[i][v], h[i][v]);
        h[i][v] = c < a.C ? h[i][v] : 0.f;
        s += h[i][v];
      }
      if (c < a.C) put_stream<R, V>(a.h, row * a.C + c, h[i]);
    }
    if (a.pre) {
      if (a.center) {
        row_sums<LANES>(s, zero, red, turn);
        mu = s * inv;
      }
      s = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          h[i][v] = (i * LANES + lane) * V < a.C ? h[i][v] - mu : 0.f;
          s = fmaf(h[i][v], h[i][v], s);
        }
      row_sums<LANES>(s, zero, red, turn);
      r2 = 1.f / sqrtf(fmaf(s, inv, a.eps));
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * LANES + lane) * V;
        float o[V];
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = fmaf(h[i][v] * r2, w[i][v], wb[i][v]);
        if (c < a.C) store_pack(static_cast<T*>(a.y) + row * a.C + c, o);
      }
    }
    if (a.stats != nullptr && lane == 0)
      *reinterpret_cast<float4*>(a.stats + 4 * row) = float4{mu1, r1, mu, r2};
  }
}

template <typename T, typename R, int LANES, int NV, int V>
__global__ __launch_bounds__((Res<LANES>::kBlock)) void res_bwd_kernel(ResArgs a,
                                                                               ResPlan p) {
  using P = Res<LANES>;
  __shared__ float red[2][kRowWaves<LANES>][2];
  __shared__ float sum[LANES > 64 ? 1 : kThreads / 64][64];
  const int lane = threadIdx.x % LANES, wave = LANES > 64 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Walk k = walk_of(a, p);
  const float inv = 1.f / (float)a.C;
  int turn = 0;  // of row_sums
  const bool row_gate = a.gate != nullptr && a.gate_rows == 1;
  float pw[NV][V], pb[NV][V], w[NV][V], gate[NV][V];
  float dpw[NV][V], dpb[NV][V], dw[NV][V], db[NV][V], dg[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * LANES + lane) * V, at = c < a.C ? c : a.C;
    parameter(a.post_w, at, a.C, a.w_bf16, a.offset, 1.f, pw[i]);
    parameter(a.post_b, at, a.C, a.w_bf16, 0.f, 0.f, pb[i]);
    parameter(a.pre_w, at, a.C, a.w_bf16, a.offset, 1.f, w[i]);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      gate[i][v] = 1.f;
      dpw[i][v] = dpb[i][v] = dw[i][v] = db[i][v] = dg[i][v] = 0.f;
    }
  }
  Raw<T, V> xn[NV], yn[NV];  // the next row
  Raw<R, V> rn[NV], hn[NV];
  RawGate<V> gn[NV];
  float4 sn;
  auto fetch = [&](int64_t row, int64_t stop) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * LANES + lane) * V;
      const bool there = row < stop;
      xn[i].load(row_of<T>(a.x, row, a.x_stride, a.C, there), c);
      rn[i].load(row_of<R>(a.r, row, a.r_stride, a.C, there && a.pre), c);
      yn[i].load(row_of<T>(a.dy, row, a.C, a.C, there && a.pre), c);
      hn[i].load(row_of<R>(a.dh, row, a.C, a.C, there && a.dh != nullptr), c);
      if (row_gate && there) gn[i].load(a, row, c);
    }
    sn = *reinterpret_cast<const float4*>(a.stats + 4 * (row < stop ? row : stop - 1));
  };
  // The workgroup's sum of one value a lane, in the first wave (or, where the
  // workgroup walks as one, in every lane's own).
  auto over_waves = [&](float x) __attribute__((always_inline)) {
    if constexpr (LANES <= 64) {
      lds_barrier();
      sum[wave][lane] = x;
      lds_barrier();
      x = (sum[0][lane] + sum[1][lane]) + (sum[2][lane] + sum[3][lane]);
    }
    return x;
  };
  const int64_t per = a.gate_rows > 1 ? a.gate_rows : a.rows;
  // one gate row at a time (all of them, where the gate has a row of its own
  // for every row)
  for (int64_t start = k.first; start < k.last;) {
    const int64_t g = start / per;
    const int64_t stop = (g + 1) * per < k.last ? (g + 1) * per : k.last;
    if (a.gate != nullptr && !row_gate) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * LANES + lane) * V;
        RawGate<V> raw;
        raw.load(a, g, c);
        raw.get(a, gate[i]);
      }
    }
    if constexpr (kAhead<LANES, V>) fetch(start + wave, stop);
    for (int64_t row = start + wave; row < stop; row += P::kWalkers) {
      float n[NV][V], h[NV][V], xh[NV][V], dy[NV][V], d[NV][V];
      if constexpr (!kAhead<LANES, V>) fetch(row, stop);
      const float mu1 = sn.x, r1 = sn.y, mu2 = sn.z, r2 = sn.w;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        xn[i].get(xh[i]);
        rn[i].get(h[i]);
        yn[i].get(dy[i]);
        hn[i].get(d[i]);
        if (row_gate) gn[i].get(a, gate[i]);
      }
      if constexpr (kAhead<LANES, V>) fetch(row + P::kWalkers, stop);
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const bool ok = (i * LANES + lane) * V < a.C;
          if (a.post) {
            xh[i][v] = ok ? (xh[i][v] - mu1) * r1 : 0.f;
            n[i][v] = fmaf(xh[i][v], pw[i][v], pb[i][v]);
          } else {
            n[i][v] = xh[i][v];
          }
        }
      if (a.pre) {
        float se = 0.f, sx = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const bool ok = (i * LANES + lane) * V < a.C;
            h[i][v] = fmaf(a.alpha * gate[i][v], n[i][v], h[i][v]);
            h[i][v] = ok ? (h[i][v] - mu2) * r2 : 0.f;
            dw[i][v] = fmaf(dy[i][v], h[i][v], dw[i][v]);
            db[i][v] += dy[i][v];
            dy[i][v] *= w[i][v];
            se += dy[i][v];
            sx = fmaf(dy[i][v], h[i][v], sx);
          }
        row_sums<LANES>(se, sx, red, turn);
        se = a.center ? se * inv : 0.f;
        sx *= inv;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int v = 0; v < V; ++v)
            d[i][v] = fmaf(r2, dy[i][v] - se - h[i][v] * sx, d[i][v]);
      }
      float se = 0.f, sx = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * LANES + lane) * V;
        if (c < a.C) put_stream<R, V>(a.dr, row * a.C + c, d[i]);
        float og[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float ad = c < a.C ? a.alpha * d[i][v] : 0.f;
          og[v] = ad * n[i][v];
          dg[i][v] += og[v];
          d[i][v] = ad * gate[i][v];
          if (a.post) {
            dpw[i][v] = fmaf(d[i][v], xh[i][v], dpw[i][v]);
            dpb[i][v] += d[i][v];
            d[i][v] *= pw[i][v];
            se += d[i][v];
            sx = fmaf(d[i][v], xh[i][v], sx);
          }
        }
        if (row_gate && a.dgate != nullptr && c < a.C) {
          if (a.gate_bf16)
            store_pack(static_cast<bf16*>(a.dgate) + row * a.C + c, og);
          else
            put_stream<float, V>(a.dgate, row * a.C + c, og);
        }
      }
      if (a.post) {
        row_sums<LANES>(se, sx, red, turn);
        se = a.center ? se * inv : 0.f;
        sx *= inv;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int v = 0; v < V; ++v) d[i][v] = r1 * (d[i][v] - se - xh[i][v] * sx);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * LANES + lane) * V;
        if (c < a.C) store_pack(static_cast<T*>(a.dx) + row * a.C + c, d[i]);
      }
    }
    if (a.dgate != nullptr && !row_gate) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float s = over_waves(dg[i][v]);
          dg[i][v] = 0.f;
          const int c = (i * LANES + lane) * V + v;
          if (wave == 0 && c < a.C) {
            if (p.per_gate > 1)
              a.gate_part[(int64_t)blockIdx.x * a.C + c] = s;
            else
              st_weight(a.dgate, g * a.C + c, s, a.gate_bf16);
          }
        }
    }
    start = stop;
  }
  if (a.part == nullptr) return;
  float* const part = a.part + (int64_t)blockIdx.x * 4 * a.C;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (i * LANES + lane) * V + v;
      const float s[4] = {over_waves(dpw[i][v]), over_waves(dpb[i][v]), over_waves(dw[i][v]),
                          over_waves(db[i][v])};
      if (wave == 0 && c < a.C)
#pragma unroll
        for (int j = 0; j < 4; ++j) part[(int64_t)j * a.C + c] = s[j];
    }
}

// Sums of the partial rows: blockIdx.y 0 .. 3 the weights', then the gate rows'.
__global__ __launch_bounds__(kThreads) void res_sums(ResArgs a, ResPlan p, int gates_from) {
  const int tc = threadIdx.x % kSumCols;
  const int64_t c = (int64_t)blockIdx.x * kSumCols + tc;
  const int64_t j = blockIdx.y;
  if (j < gates_from) {
    void* const to[4] = {a.dpost_w, a.dpost_b, a.dpre_w, a.dpre_b};
    if (to[j] == nullptr) return;  // the whole workgroup
    // rows of part are 4 C apart; columns j C ..
    const float s = column_sum(a.part + j * a.C, p.parts, 4 * (int64_t)a.C,
                               c < a.C ? c : 4 * (int64_t)a.C);
    if (threadIdx.x < kSumCols && c < a.C) st_weight(to[j], c, s, a.w_bf16);
  } else {
    const int64_t g = j - gates_from;
    const float s = column_sum(a.gate_part + g * p.per_gate * a.C, p.per_gate, a.C, c);
    if (threadIdx.x < kSumCols && c < a.C) st_weight(a.dgate, g * a.C + c, s, a.gate_bf16);
  }
}

template <typename T, typename R, bool BWD, int LANES, int NV, int V>
hipError_t go(const ResArgs& a, const ResPlan& p, hipStream_t s) {
  using P = Res<LANES>;
  if constexpr (!BWD) {
    hipLaunchKernelGGL((res_fwd_kernel<T, R, LANES, NV, V>), dim3((unsigned)p.parts),
                       dim3(P::kBlock), 0, s, a, p);
    const hipError_t e = hipGetLastError();
    note_launch(s);
    return e;
  } else {
    hipLaunchKernelGGL((res_bwd_kernel<T, R, LANES, NV, V>), dim3((unsigned)p.parts),
                       dim3(P::kBlock), 0, s, a, p);
    hipError_t e = hipGetLastError();
    note_launch(s);
    const int64_t per = a.gate_rows > 1 ? a.gate_rows : a.rows;
    const int weights = a.part != nullptr ? 4 : 0;
    const int64_t gates = a.gate_part != nullptr ? a.rows / per : 0;
    if (e != hipSuccess || weights + gates == 0) return e;
    hipLaunchKernelGGL(res_sums, dim3((a.C + kSumCols - 1) / kSumCols, (unsigned)(weights + gates)),
                       dim3(kThreads), 0, s, a, p, weights);
    e = hipGetLastError();
    note_launch(s);
    return e;
  }
}

template <typename T, typename R, bool BWD, int V>
hipError_t launch_v(const ResArgs& a, const ResPlan& p, hipStream_t s) {
  constexpr int NV = 8 / V;  // 8 channels a lane
  switch (p.lanes) {
    case 64: return go<T, R, BWD, 64, NV, V>(a, p, s);
    case 256: return go<T, R, BWD, 256, NV, V>(a, p, s);
    case 512: return go<T, R, BWD, 512, NV, V>(a, p, s);
    case 1024: return go<T, R, BWD, 1024, NV, V>(a, p, s);
  }
  return hipErrorInvalidValue;
}

template <bool BWD>
hipError_t launch(const ResArgs& a, const ResPlan& p, bool is_bf16, bool stream_f32,
                  hipStream_t s) {
  if (!is_bf16)
    return p.vec ? launch_v<float, float, BWD, 4>(a, p, s)
                 : launch_v<float, float, BWD, 1>(a, p, s);
  if (stream_f32)
    return p.vec ? launch_v<bf16, float, BWD, 8>(a, p, s) : launch_v<bf16, float, BWD, 1>(a, p, s);
  return p.vec ? launch_v<bf16, bf16, BWD, 8>(a, p, s) : launch_v<bf16, bf16, BWD, 1>(a, p, s);
}

}  // namespace

// Lanes of a row (8 channels each) and the workgroups' rows.
bool res_plan(const ResArgs& a, bool is_bf16, bool bwd, ResPlan* p) {
  const int64_t V = is_bf16 ? 8 : 4;
  p->vec = a.C % V == 0 && a.x_stride % V == 0 && a.r_stride % V == 0 && a.gate_stride % V == 0;
  const int64_t lanes = (a.C + 7) / 8;
  if (lanes > 1024) return false;
  p->lanes = lanes <= 64 ? 64 : lanes <= 256 ? 256 : lanes <= 512 ? 512 : 1024;
  const int64_t walkers = p->lanes > 64 ? 1 : kThreads / 64;
  const int64_t per = a.gate_rows > 1 ? a.gate_rows : (a.rows < 1 ? 1 : a.rows);
  int64_t want = p->lanes > 64 ? 131072 / p->lanes : 512;
  if (!bwd || !p->vec) want *= 2;
  int64_t step = (a.rows + want - 1) / want;
  if (step < walkers) step = walkers;
  if (step < per) {  // parts of a gate row
    p->per_gate = per / step;
    if (p->per_gate < 1) p->per_gate = 1;
    p->step = (per + p->per_gate - 1) / p->per_gate;
    p->per_gate = (per + p->step - 1) / p->step;  // none of them empty
    p->parts = p->per_gate * (a.rows / per);
  } else {  // whole gate rows
    p->step = step / per * per;
    p->per_gate = 1;
    p->parts = (a.rows + p->step - 1) / p->step;
  }
  if (p->parts < 1) p->parts = 1;
  return true;
}

hipError_t launch_res_fwd(const ResArgs& a, const ResPlan& p, bool is_bf16, bool stream_f32,
                          hipStream_t s) {
  return launch<false>(a, p, is_bf16, stream_f32, s);
}
hipError_t launch_res_bwd(const ResArgs& a, const ResPlan& p, bool is_bf16, bool stream_f32,
                          hipStream_t s) {
  return launch<true>(a, p, is_bf16, stream_f32, s);
}

}  // namespace gdr
