// Short causal convolution over channels-last rows on gfx950: per channel
//   s_t = bias + sum_{j<K} w[j] x_{t-(K-1)+j},   y_t = act(s_t),
// x before the sequence from the carried window (state) or zero.  The
// backward recomputes s from x:
//   ds_t = dy_t act'(s_t),  dx_t = sum_j w[j] ds_{t+(K-1)-j},
//   dw[j] = sum_t ds_t x_{t-(K-1)+j},  dbias = sum_t ds_t.
// Bound by HBM bytes: x and y once (forward), x, dy and dx once (backward).
//
// Mapping: a thread owns 16 bytes of neighbouring channels (one channel where
// rows or strides do not divide) and marches over a tile of steps with the
// last K - 1 inputs in registers, so every row is loaded once per tile plus a
// halo of K - 1 rows.
#include "gdr_layer.h"

namespace gdr {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;  // rows of one turn; the next turn's are loaded ahead

// Input row t of the sequence: x for t >= 0 (t < len), else the window, else 0.
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> input_row(const ConvArgs& a, const Span& sp, int b, int t,
                                                int c) {
  if (t >= 0)
    return load_pack<T, V>(static_cast<const T*>(a.x) + (sp.first + t) * a.x_stride + c);
  if (a.state == nullptr) return zero_pack<T, V>();
  return load_pack<T, V>(static_cast<const T*>(a.state) +
                         ((int64_t)b * (a.K - 1) + (a.K - 1 + t)) * a.C + c);
}

template <int K, int V>
__device__ __forceinline__ void load_weights(const ConvArgs& a, int c, float (&w)[V * K],
                                             float (&bias)[V]) {
  ld_weights<V * K, (V > 1)>(a.w, (int64_t)c * K, a.w_bf16, w);
  if (a.bias != nullptr) {
    ld_weights<V, (V > 1)>(a.bias, c, a.w_bf16, bias);
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) bias[v] = 0.f;
  }
}

template <typename T, int K, int V>
__global__ __launch_bounds__(kThreads) void conv_fwd_kernel(ConvArgs a, int cblocks, int steps) {
  const int c = ((blockIdx.x % cblocks) * kThreads + threadIdx.x) * V;
  const int tile = blockIdx.x / cblocks;
  const int b = blockIdx.y;
  if (c >= a.C) return;
  const Span sp = span_of(a.spans, b, a.T, a.rows);
  const int64_t t0l = (int64_t)tile * steps;
  if (t0l > 0 && t0l >= sp.len) return;
  const int t0 = (int)t0l, t1 = sp.len - t0 < steps ? sp.len : t0 + steps;

  float w[V * K], bias[V];  // weight[c + v][j] at v K + j
  load_weights<K, V>(a, c, w, bias);
  Pack<T, V> hist[K > 1 ? K - 1 : 1];
#pragma unroll
  for (int i = 0; i < K - 1; ++i) hist[i] = input_row<T, V>(a, sp, b, t0 - (K - 1) + i, c);

  // the window left behind: the last K - 1 of (window, x).  The thread that
  // read the window's channels writes them, after all its reads of it.
  if (tile == 0 && a.state_out != nullptr) {
    Pack<T, V> out[K > 1 ? K - 1 : 1];
#pragma unroll
    for (int i = 0; i < K - 1; ++i) out[i] = input_row<T, V>(a, sp, b, sp.len - (K - 1) + i, c);
    T* const o = static_cast<T*>(a.state_out) + (int64_t)b * (K - 1) * a.C + c;
#pragma unroll
    for (int i = 0; i < K - 1; ++i)
      *reinterpret_cast<Pack<T, V>*>(o + (int64_t)i * a.C) = out[i];
  }

  const T* xp = static_cast<const T*>(a.x) + (sp.first + t0) * a.x_stride + c;
  T* yp = static_cast<T*>(a.y) + (sp.first + t0) * a.C + c;
  // rows t .. t + kUnroll - 1, clamped to the tile's last one
  auto fetch = [&](int t, Pack<T, V>(&in)[kUnroll]) __attribute__((always_inline)) {
#pragma unroll
    for (int r = 0; r < kUnroll; ++r) {
      const int at = t + r < t1 ? t + r : t1 - 1;
      in[r] = load_pack<T, V>(xp + (int64_t)(at - t0) * a.x_stride);
    }
  };
  float win[K][V];  // win[K - 1]: the current input
#pragma unroll
  for (int i = 0; i < K - 1; ++i) unpack(hist[i], win[i]);
  Pack<T, V> next[kUnroll];
  if (t0 < t1) fetch(t0, next);
  for (int t = t0; t < t1; t += kUnroll) {
    Pack<T, V> in[kUnroll];
#pragma unroll
    for (int r = 0; r < kUnroll; ++r) in[r] = next[r];
    if (t + kUnroll < t1) fetch(t + kUnroll, next);
#pragma unroll
    for (int r = 0; r < kUnroll; ++r) {
      unpack(in[r], win[K - 1]);
      float s[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        s[v] = bias[v];
#pragma unroll
        for (int j = 0; j < K; ++j) s[v] = fmaf(w[v * K + j], win[j][v], s[v]);
        if (a.act) s[v] = silu(s[v]);
#pragma unroll
        for (int j = 0; j + 1 < K; ++j) win[j][v] = win[j + 1][v];
      }
      if (t + r < t1) store_pack(yp + (int64_t)r * a.C, s);
    }
    yp += (int64_t)kUnroll * a.C;
  }
}

// Backward: wave q of a workgroup takes steps [t0, t1) of its channels (64
// lanes) and adds its dw, dbias over the workgroup's four waves in LDS, so
// that one partial sum per four tiles reaches memory.
template <typename T, int K, int V>
__global__ __launch_bounds__(kThreads) void conv_bwd_kernel(ConvArgs a, int cblocks, int steps) {
  __shared__ float red[3][K + 1][V][64];
  const int lane = threadIdx.x & 63, q = threadIdx.x >> 6;
  const int c = ((blockIdx.x % cblocks) * 64 + lane) * V;
  const int group = blockIdx.x / cblocks;
  const int b = blockIdx.y;
  const bool cok = c < a.C;
  const int cc = cok ? c : 0;
  const Span sp = span_of(a.spans, b, a.T, a.rows);
  const int64_t t0l = ((int64_t)group * 4 + q) * steps;
  const bool first = t0l == 0;
  const bool any = cok && (first || t0l < sp.len);

  float dw[K][V], db[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    db[v] = 0.f;
#pragma unroll
    for (int j = 0; j < K; ++j) dw[j][v] = 0.f;
  }
  if (any) {
    const int t0 = (int)t0l, t1 = sp.len - t0 < steps ? sp.len : t0 + steps;
    float w[V * K], bias[V];
    load_weights<K, V>(a, cc, w, bias);
    float win[K][V], ds[K][V];  // the inputs and ds of the last K steps
#pragma unroll
    for (int i = 0; i < K - 1; ++i) unpack(input_row<T, V>(a, sp, b, t0 - (K - 1) + i, cc), win[i]);
#pragma unroll
    for (int i = 0; i < K; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) ds[i][v] = 0.f;
    const T* const xb = static_cast<const T*>(a.x) + sp.first * a.x_stride + cc;
    const T* const dyb = static_cast<const T*>(a.dy) + sp.first * a.C + cc;
    T* const dxb = static_cast<T*>(a.dx) + sp.first * a.C + cc;
    // step t forms ds_t and completes dx of step t - (K - 1); the last K - 1
    // steps only complete.  Rows from sp.len on count as ds = 0.
    const int tend = t1 + K - 1;
    Pack<T, V> nx[kUnroll], nd[kUnroll];
    auto fetch = [&](int t) __attribute__((always_inline)) {
#pragma unroll
      for (int r = 0; r < kUnroll; ++r) {
        const int tt = t + r < sp.len ? t + r : sp.len - 1;  // -1: an empty sequence
        nx[r] = tt < 0 ? zero_pack<T, V>() : load_pack<T, V>(xb + (int64_t)tt * a.x_stride);
        nd[r] = tt < 0 ? zero_pack<T, V>() : load_pack<T, V>(dyb + (int64_t)tt * a.C);
      }
    };
    fetch(t0);
    for (int t = t0; t < tend; t += kUnroll) {
      Pack<T, V> in[kUnroll], dyv[kUnroll];
#pragma unroll
      for (int r = 0; r < kUnroll; ++r) {
        in[r] = nx[r];
        dyv[r] = nd[r];
      }
      if (t + kUnroll < tend) fetch(t + kUnroll);
#pragma unroll
      for (int r = 0; r < kUnroll; ++r) {
        const int tt = t + r;
        if (tt >= tend) continue;
        float dyf[V], out[V];
        unpack(in[r], win[K - 1]);
        unpack(dyv[r], dyf);
        const bool mine = tt < t1;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float d = dyf[v];
          if (a.act) {
            float s = bias[v];
#pragma unroll
            for (int j = 0; j < K; ++j) s = fmaf(w[v * K + j], win[j][v], s);
            d *= dsilu(s, sigmoid(s));
          }
          if (tt >= sp.len) d = 0.f;
#pragma unroll
          for (int j = 0; j + 1 < K; ++j) ds[j][v] = ds[j + 1][v];
          ds[K - 1][v] = d;
          if (mine) {
            db[v] += d;
#pragma unroll
            for (int j = 0; j < K; ++j) dw[j][v] = fmaf(d, win[j][v], dw[j][v]);
          }
          out[v] = 0.f;
#pragma unroll
          for (int j = 0; j < K; ++j) out[v] = fmaf(w[v * K + j], ds[K - 1 - j][v], out[v]);
#pragma unroll
          for (int j = 0; j + 1 < K; ++j) win[j][v] = win[j + 1][v];
        }
        const int to = tt - (K - 1);  // the input whose gradient is complete
        if (to < t0 && !first) continue;
        if (a.dstate_out != nullptr && to >= sp.len - (K - 1)) {
          float e[V];
          unpack(load_pack<T, V>(static_cast<const T*>(a.dstate_out) +
                                 ((int64_t)b * (K - 1) + (to - (sp.len - (K - 1)))) * a.C + cc),
                 e);
#pragma unroll
          for (int v = 0; v < V; ++v) out[v] += e[v];
        }
        if (to >= 0)
          store_pack(dxb + (int64_t)to * a.C, out);
        else if (a.dstate != nullptr)
          store_pack(static_cast<T*>(a.dstate) + ((int64_t)b * (K - 1) + (K - 1 + to)) * a.C + cc,
                     out);
      }
    }
  }
  if (q > 0) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      red[q - 1][K][v][lane] = db[v];
#pragma unroll
      for (int j = 0; j < K; ++j) red[q - 1][j][v][lane] = dw[j][v];
    }
  }
  __syncthreads();
  if (q == 0 && cok) {
    const int64_t part = (int64_t)b * (gridDim.x / cblocks) + group;
    float* const p = a.part + part * (K + 1) * a.C + cc;
#pragma unroll
    for (int j = 0; j <= K; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float own = j < K ? dw[j < K ? j : 0][v] : db[v];
        p[(int64_t)j * a.C + v] =
            own + red[0][j][v][lane] + red[1][j][v][lane] + red[2][j][v][lane];
      }
  }
}

struct ConvSumStore {
  void* dw;
  void* dbias;
  int C, K, w_bf16;
  __device__ void operator()(int64_t i, float x) const {
    const int j = (int)(i / C), c = (int)(i % C);
    if (j < K)
      st_weight(dw, (int64_t)c * K + j, x, w_bf16);
    else if (dbias != nullptr)
      st_weight(dbias, c, x, w_bf16);
  }
};

template <typename T>
bool vectors(const ConvArgs& a) {
  constexpr int V = 16 / sizeof(T);
  return a.C % V == 0 && a.x_stride % V == 0;
}

template <typename T, int K, int V>
hipError_t fwd(const ConvArgs& a, hipStream_t s) {
  const int cblocks = (a.C + kThreads * V - 1) / (kThreads * V);
  // 16 to 32 steps a tile, by what gives 256 compute units eight waves each:
  // shorter tiles read more of the halo, longer ones leave fewer loads in
  // flight (7 packed prompts of 6000 rows, 14336 channels: 72 us at 16 steps,
  // 78 at 48; one sequence of 2048: 27 us at 28 steps, 30 at 16, 32 at 48)
  const int64_t waves = (int64_t)cblocks * (kThreads / 64) * a.B;
  int64_t steps = waves * a.T / 2048;
  steps = steps < 16 ? 16 : (steps > 32 ? 32 : steps);
  int64_t tiles = (a.T + steps - 1) / steps;
  while (tiles * cblocks > INT32_MAX) {
    steps *= 2;
    tiles = (a.T + steps - 1) / steps;
  }
  if (tiles < 1) tiles = 1;
  hipLaunchKernelGGL((conv_fwd_kernel<T, K, V>), dim3((unsigned)(tiles * cblocks), a.B),
                     dim3(kThreads), 0, s, a, cblocks, (int)steps);
  const hipError_t e = hipGetLastError();
  note_launch(s);
  return e;
}

template <typename T, int K, int V>
hipError_t bwd(const ConvArgs& a, hipStream_t s) {
  const int cblocks = (a.C + 64 * V - 1) / (64 * V);
  const int steps = conv_bwd_steps(a.B, a.T, a.C);
  const int64_t parts = conv_bwd_parts(a.B, a.T, a.C);
  hipLaunchKernelGGL((conv_bwd_kernel<T, K, V>), dim3((unsigned)(parts / a.B * cblocks), a.B),
                     dim3(kThreads), 0, s, a, cblocks, steps);
  hipError_t e = hipGetLastError();
  note_launch(s);
  if (e != hipSuccess) return e;
  return launch_column_sums(a.part, parts, (int64_t)(K + 1) * a.C,
                            ConvSumStore{a.dw, a.dbias, a.C, K, a.w_bf16}, s);
}

template <typename T, bool BWD, int K>
hipError_t launch_v(const ConvArgs& a, hipStream_t s) {
  constexpr int V = 16 / sizeof(T);
  // the backward holds 4 K + 2 values per channel: four channels a thread
  // in either type (bf16: 8 bytes a load, 47.8 us against 66.5 with 16 bytes,
  // 236 registers and two waves a SIMD)
  if (vectors<T>(a)) return BWD ? bwd<T, K, 4>(a, s) : fwd<T, K, V>(a, s);
  return BWD ? bwd<T, K, 1>(a, s) : fwd<T, K, 1>(a, s);
}

template <typename T, bool BWD>
hipError_t launch_k(const ConvArgs& a, hipStream_t s) {
  switch (a.K) {
    case 1: return launch_v<T, BWD, 1>(a, s);
    case 2: return launch_v<T, BWD, 2>(a, s);
    case 3: return launch_v<T, BWD, 3>(a, s);
    case 4: return launch_v<T, BWD, 4>(a, s);
    case 5: return launch_v<T, BWD, 5>(a, s);
    case 6: return launch_v<T, BWD, 6>(a, s);
    case 7: return launch_v<T, BWD, 7>(a, s);
    case 8: return launch_v<T, BWD, 8>(a, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace

// 16 steps a wave, 32 where that still leaves 4096 waves (the halo and the
// partial sums halve): 2048 rows of 14336 bf16 channels take 44.6 us at 16,
// 45.8 at 32, 50.7 at 48.  Sized for 256 compute units and vector loads: it
// sizes a workspace too, which must not depend on the current device or on
// strides.
int conv_bwd_steps(int64_t B, int64_t T, int64_t C) {
  const int64_t waves = (C + 255) / 256 * B;
  int64_t steps = waves * T / 32 >= 4096 ? 32 : 16;
  // the grid's x dimension holds (tiles / 4) x (channel blocks, at most one
  // per 64 channels)
  while ((T + 4 * steps - 1) / (4 * steps) * ((C + 63) / 64) > INT32_MAX) steps *= 2;
  return (int)steps;
}

int64_t conv_bwd_parts(int64_t B, int64_t T, int64_t C) {
  const int64_t steps = 4 * (int64_t)conv_bwd_steps(B, T, C);
  const int64_t groups = (T + steps - 1) / steps;
  return B * (groups < 1 ? 1 : groups);
}

hipError_t launch_conv_fwd(const ConvArgs& a, bool is_bf16, hipStream_t s) {
  return is_bf16 ? launch_k<bf16, false>(a, s) : launch_k<float, false>(a, s);
}
hipError_t launch_conv_bwd(const ConvArgs& a, bool is_bf16, hipStream_t s) {
  return is_bf16 ? launch_k<bf16, true>(a, s) : launch_k<float, true>(a, s);
}

}  // namespace gdr
