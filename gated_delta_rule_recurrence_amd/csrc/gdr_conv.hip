// Short causal convolution over channels-last rows on gfx950: per channel
//   s_t = bias + sum_{j<K} w[j] x_{t-(K-1)+j},   y_t = act(s_t),
// x before the sequence from the carried window (state) or zero.  The
// backward recomputes s from x:
//   ds_t = dy_t act'(s_t),  dx_t = sum_j w[j] ds_{t+(K-1)-j},
//   dw[j] = sum_t ds_t x_{t-(K-1)+j},  dbias = sum_t ds_t.
// Bound by HBM bytes: x and y once (forward), x, dy and dx once (backward).
// Measured (bf16, 14336 channels, K = 4; a large copy reaches 4.98 TB/s):
// forward over 6000 packed rows 76 us, 4.5 TB/s; over 2048 rows 27 us, 4.4
// TB/s; backward over those 39 to 43 us, 4.1 to 4.5 TB/s, and 5 us for the sums
// of dw.
//
// Mapping: a thread owns 16 bytes of neighbouring channels (8 in the backward;
// one channel where rows or strides do not divide) and marches over a tile of
// steps with the last K - 1 inputs in registers, so every row is loaded once
// per tile plus a halo of K - 1 rows.  A row is a buffer whose bound is its
// end, or nothing where there is no such row: no load and no store has a
// branch around it, and the first loads go out together (one token for 64
// requests: 5.4 us, of which two trips to memory, spans and then the rest,
// and the launch are most; 14.7 with a wait between each kind).
#include "gdr_layer.h"

namespace gdr {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;  // rows of one turn

// Input row t of the sequence: x for 0 <= t < end, the window for t < 0, else
// a row of no bytes, read as zeros.  t is the same for the whole wave; the
// choices are between integers, which the compiler keeps in scalar registers
// (a choice between conditions goes through vector registers, and every load
// then becomes a loop over its lanes).
template <typename T>
__device__ __forceinline__ Buffer input_row(const ConvArgs& a, const Span& sp, int b, int t,
                                            int end) {
  constexpr int64_t kSize = sizeof(T);
  const int row = a.C * (int)kSize;
  const int inside = (t - end) >> 31 & row, carried = a.state != nullptr ? row : 0;
  const char* const x = static_cast<const char*>(a.x) + (sp.first + t) * a.x_stride * kSize;
  const char* const s =
      static_cast<const char*>(a.state) + ((int64_t)b * (a.K - 1) + (a.K - 1 + t)) * row;
  return buffer_of(t >= 0 ? x : s, 0, t >= 0 ? inside : carried);
}
// A walk over rows: row r from here on, of no bytes unless r < left.
struct Rows {
  const char* p;
  int64_t step;  // bytes from row to row
  int row;       // bytes of one
  __device__ __forceinline__ Buffer at(int r, int left) const {
    return buffer_of(p, r * step, (r - left) >> 31 & row);
  }
  __device__ __forceinline__ void advance(int rows) { p += rows * step; }
};
// From row t of the sequence, in x or in a dense tensor
template <typename T>
__device__ __forceinline__ Rows rows_of(const ConvArgs& a, const void* p, int64_t stride,
                                        const Span& sp, int t) {
  const int64_t step = stride * (int64_t)sizeof(T);
  return Rows{static_cast<const char*>(p) + (sp.first + t) * step, step, a.C * (int)sizeof(T)};
}
template <typename T, int V>
__device__ __forceinline__ void put_pack(Buffer b, uint32_t offset, const Pack<T, V>& x) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  constexpr int kBytes = V * sizeof(T);
  if constexpr (kBytes == 2)
    __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, x), b.resource(),
                                          (int)offset, 0, 0);
  else if constexpr (kBytes == 4)
    __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, x), b.resource(),
                                          (int)offset, 0, 0);
  else if constexpr (kBytes == 8)
    __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, x), b.resource(), (int)offset,
                                          0, 0);
  else
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), b.resource(), (int)offset,
                                           0, 0);
}
// The sequence's rows, in scalar registers.
__device__ __forceinline__ Span uniform_span(const ConvArgs& a, int b) {
  Span sp = span_of(a.spans, b, a.T, a.rows);
  sp.first = __builtin_amdgcn_readfirstlane((int)sp.first);
  sp.len = __builtin_amdgcn_readfirstlane(sp.len);
  return sp;
}

// U rows of one turn (the next turn's are loaded ahead).
template <typename T, int K, int V, int U>
__global__ __launch_bounds__(kThreads) void conv_fwd_kernel(ConvArgs a, int cblocks, int steps) {
  const int tile = __builtin_amdgcn_readfirstlane((int)(blockIdx.x / cblocks));
  const int c = ((int)(blockIdx.x - (uint32_t)tile * cblocks) * kThreads + (int)threadIdx.x) * V;
  const int b = blockIdx.y;
  if (c >= a.C) return;
  const Span sp = uniform_span(a, b);
  const int64_t t0l = (int64_t)tile * steps;
  if (t0l > 0 && t0l >= sp.len) return;
  const int t0 = (int)t0l, t1 = sp.len - t0 < steps ? sp.len : t0 + steps;
  const uint32_t oc = (uint32_t)c * (uint32_t)sizeof(T);

  // all the first loads before any use: the rows before the tile, its first
  // rows, the weights, and (the first tile) the window left behind
  Pack<T, V> hist[K > 1 ? K - 1 : 1], next[U], last[K > 1 ? K - 1 : 1];
#pragma unroll
  for (int i = 0; i < K - 1; ++i)
    hist[i] = get_pack<T, V>(input_row<T>(a, sp, b, t0 - (K - 1) + i, sp.len), oc);
  Rows xs = rows_of<T>(a, a.x, a.x_stride, sp, t0), ys = rows_of<T>(a, a.y, a.C, sp, t0);
#pragma unroll
  for (int r = 0; r < U; ++r) next[r] = get_pack<T, V>(xs.at(r, t1 - t0), oc);
  Weights<V * K, (V > 1)> wr;
  Weights<V, (V > 1)> br;
  wr.load(a.w, (int64_t)c * K, (int64_t)a.C * K, a.w_bf16);
  br.load(a.bias, c, a.C, a.w_bf16);
  const bool leave = tile == 0 && a.state_out != nullptr;
  if (leave && U > 1)  // (of a single token they are those rows, one on)
#pragma unroll
    for (int i = 0; i < K - 1; ++i)
      last[i] = get_pack<T, V>(input_row<T>(a, sp, b, sp.len - (K - 1) + i, sp.len), oc);
  float w[V * K], bias[V];  // weight[c + v][j] at v K + j
  wr.get(a.w_bf16, w);
  br.get(a.w_bf16, bias);
  // the last K - 1 of (window, x).  The thread that read the window's
  // channels writes them, after all its reads of it: state_out may be state.
  if (leave) {
    const int64_t size = a.C * (int64_t)sizeof(T);
#pragma unroll
    for (int i = 0; i < K - 1; ++i) {
      if (U == 1) {
        const Pack<T, V> on = i + 2 < K ? hist[i + 2 < K ? i + 1 : 0] : next[0];
        last[i] = sp.len > 0 ? on : hist[i];
      }
      put_pack(buffer_of(a.state_out, ((int64_t)b * (K - 1) + i) * size, size), oc, last[i]);
    }
  }

  float win[K][V];  // win[K - 1]: the current input
#pragma unroll
  for (int i = 0; i < K - 1; ++i) unpack(hist[i], win[i]);
  for (int t = t0; t < t1; t += U) {
    Pack<T, V> in[U];
#pragma unroll
    for (int r = 0; r < U; ++r) in[r] = next[r];
    const int left = t1 - t;
    xs.advance(U);
    if (left > U)
#pragma unroll
      for (int r = 0; r < U; ++r) next[r] = get_pack<T, V>(xs.at(r, left - U), oc);
#pragma unroll
    for (int r = 0; r < U; ++r) {
      unpack(in[r], win[K - 1]);
      float s[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        s[v] = bias[v];
#pragma unroll
        for (int j = 0; j < K; ++j) s[v] = fmaf(w[v * K + j], win[j][v], s[v]);
#pragma unroll
        for (int j = 0; j + 1 < K; ++j) win[j][v] = win[j + 1][v];
      }
      if (a.act)
#pragma unroll
        for (int v = 0; v < V; ++v) s[v] = silu(s[v]);
      Pack<T, V> out;
      pack(s, out);
      put_pack(ys.at(r, left), oc, out);
    }
    ys.advance(U);
  }
}

// Backward: wave q of a workgroup takes steps [t0, t1) of its channels (64
// lanes) and adds its dw, dbias over the workgroup's four waves in LDS, so
// that one partial sum per four tiles reaches memory.
template <typename T, int K, int V>
__global__ __launch_bounds__(kThreads) void conv_bwd_kernel(ConvArgs a, int cblocks, int steps) {
  __shared__ float red[3][K + 1][V][64];
  const int lane = threadIdx.x & 63, q = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = __builtin_amdgcn_readfirstlane((int)(blockIdx.x / cblocks));
  const int c = ((int)(blockIdx.x - (uint32_t)group * cblocks) * 64 + lane) * V;
  const int b = blockIdx.y;
  const bool cok = c < a.C;
  const int cc = cok ? c : 0;
  const Span sp = uniform_span(a, b);
  const int64_t t0l = ((int64_t)group * 4 + q) * steps;
  const bool first = t0l == 0;
  // (numbered through the pieces: a workgroup past the sequence has no sums)
  if (a.packed && group > 0 && (int64_t)group * 4 * steps >= sp.len) return;
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
    const uint32_t oc = (uint32_t)cc * (uint32_t)sizeof(T);
    Pack<T, V> hist[K > 1 ? K - 1 : 1], nx[kUnroll], nd[kUnroll];
#pragma unroll
    for (int i = 0; i < K - 1; ++i)
      hist[i] = get_pack<T, V>(input_row<T>(a, sp, b, t0 - (K - 1) + i, sp.len), oc);
    Rows xs = rows_of<T>(a, a.x, a.x_stride, sp, t0), dys = rows_of<T>(a, a.dy, a.C, sp, t0);
    Rows dxs = rows_of<T>(a, a.dx, a.C, sp, t0);
    auto fetch = [&](int left) __attribute__((always_inline)) {
#pragma unroll
      for (int r = 0; r < kUnroll; ++r) {
        nx[r] = get_pack<T, V>(xs.at(r, left), oc);
        nd[r] = get_pack<T, V>(dys.at(r, left), oc);
      }
      xs.advance(kUnroll);
      dys.advance(kUnroll);
    };
    fetch(sp.len - t0);
    Weights<V * K, (V > 1)> wr;
    Weights<V, (V > 1)> br;
    wr.load(a.w, (int64_t)cc * K, (int64_t)a.C * K, a.w_bf16);
    br.load(a.bias, cc, a.C, a.w_bf16);
    float w[V * K], bias[V];
    wr.get(a.w_bf16, w);
    br.get(a.w_bf16, bias);
    float win[K][V], ds[K][V];  // the inputs and ds of the last K steps
#pragma unroll
    for (int i = 0; i < K - 1; ++i) unpack(hist[i], win[i]);
#pragma unroll
    for (int i = 0; i < K; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) ds[i][v] = 0.f;
    // step t forms ds_t and completes dx of step t - (K - 1); the last K - 1
    // steps only complete.  Rows from sp.len on count as ds = 0.
    const int tend = t1 + K - 1;
    for (int t = t0; t < tend; t += kUnroll) {
      Pack<T, V> in[kUnroll], dyv[kUnroll];
#pragma unroll
      for (int r = 0; r < kUnroll; ++r) {
        in[r] = nx[r];
        dyv[r] = nd[r];
      }
      if (t + kUnroll < tend) fetch(sp.len - (t + kUnroll));
#pragma unroll
      for (int r = 0; r < kUnroll; ++r) {
        const int tt = t + r;
        if (tt >= tend) continue;
        float dyf[V], out[V];
        unpack(in[r], win[K - 1]);
        unpack(dyv[r], dyf);
        const bool mine = tt < t1;
        if (a.act)
#pragma unroll
          for (int v = 0; v < V; ++v) {
            float s = bias[v];
#pragma unroll
            for (int j = 0; j < K; ++j) s = fmaf(w[v * K + j], win[j][v], s);
            dyf[v] *= dsilu(s, sigmoid(s));
          }
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float d = tt < sp.len ? dyf[v] : 0.f;
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
        const int64_t size = a.C * (int64_t)sizeof(T);
        if (a.dstate_out != nullptr && to >= sp.len - (K - 1)) {
          float e[V];
          const int64_t i = (int64_t)b * (K - 1) + (to - (sp.len - (K - 1)));
          unpack(get_pack<T, V>(buffer_of(a.dstate_out, i * size, size), oc), e);
#pragma unroll
          for (int v = 0; v < V; ++v) out[v] += e[v];
        }
        Pack<T, V> o;
        pack(out, o);
        if (to >= 0)
          put_pack(dxs.at(r - (K - 1), sp.len - t), oc, o);
        else if (a.dstate != nullptr)
          put_pack(buffer_of(a.dstate, ((int64_t)b * (K - 1) + (K - 1 + to)) * size, size), oc, o);
      }
      dxs.advance(kUnroll);
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
  if (q > 0) return;
  int64_t part = (int64_t)b * (gridDim.x / cblocks) + group;
  if (a.packed) {
    part = pieces_before(a.spans, b, a.T, a.rows, 4 * steps) + group;
    if (sp.len == 0 || part >= a.parts) return;  // (parts: of sequences that overlap)
  }
  if (cok) {
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

// dw and dbias from the partial sums.
__global__ __launch_bounds__(kThreads) void conv_sums(ConvArgs a) {
  int64_t parts = a.parts;
  if (a.packed) {
    const int64_t used = pieces_before(a.spans, a.B, a.T, a.rows, 4 * a.steps);
    parts = used < parts ? used : parts;
  }
  const int64_t i = (int64_t)blockIdx.x * kSumCols + threadIdx.x % kSumCols;
  const int64_t width = (int64_t)(a.K + 1) * a.C;
  const float x = column_sum(a.part, parts, width, i);
  if (threadIdx.x >= kSumCols || i >= width) return;
  const int j = (int)(i / a.C), c = (int)(i % a.C);
  if (j < a.K)
    st_weight(a.dw, (int64_t)c * a.K + j, x, a.w_bf16);
  else if (a.dbias != nullptr)
    st_weight(a.dbias, c, x, a.w_bf16);
}

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
  steps = steps < kConvTile ? kConvTile : (steps > 32 ? 32 : steps);
  int64_t tiles = (a.T + steps - 1) / steps;
  while (tiles * cblocks > kMaxGrid) {
    steps *= 2;
    tiles = (a.T + steps - 1) / steps;
  }
  if (tiles < 1) tiles = 1;
  // single tokens: a turn of one row (64 requests: 5.6 us, 6.8 with the
  // arithmetic of four; a test for the end within the turn costs prompts 2.5%)
  const dim3 grid((unsigned)(tiles * cblocks), a.B);
  if (a.T == 1)
    hipLaunchKernelGGL((conv_fwd_kernel<T, K, V, 1>), grid, dim3(kThreads), 0, s, a, cblocks,
                       (int)steps);
  else
    hipLaunchKernelGGL((conv_fwd_kernel<T, K, V, kUnroll>), grid, dim3(kThreads), 0, s, a, cblocks,
                       (int)steps);
  const hipError_t e = hipGetLastError();
  note_launch(s);
  return e;
}

// Workgroups along a sequence, at least one: four waves of `steps` each.
int64_t conv_groups(int64_t T, int64_t steps) {
  const int64_t groups = (T + 4 * steps - 1) / (4 * steps);
  return groups < 1 ? 1 : groups;
}

template <typename T, int K, int V>
hipError_t bwd(const ConvArgs& a, hipStream_t s) {
  const int cblocks = (a.C + 64 * V - 1) / (64 * V);
  hipLaunchKernelGGL((conv_bwd_kernel<T, K, V>),
                     dim3((unsigned)(conv_groups(a.T, a.steps) * cblocks), a.B), dim3(kThreads), 0,
                     s, a, cblocks, a.steps);
  hipError_t e = hipGetLastError();
  note_launch(s);
  if (e != hipSuccess) return e;
  const int64_t blocks = ((int64_t)(K + 1) * a.C + kSumCols - 1) / kSumCols;
  hipLaunchKernelGGL(conv_sums, dim3((unsigned)blocks), dim3(kThreads), 0, s, a);
  e = hipGetLastError();
  note_launch(s);
  return e;
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

// 16 steps a wave, 32 where that still leaves two waves a SIMD (the halo and
// the partial sums halve).  A backward pass in us at 16 / 32 steps, by the
// waves that 32 leave (bf16, 14336 or 4096 channels): 1792 26.7 / 27.3, 2048
// 26.6 / 26.6, 2576 35.3 / 32.0, 3024 37.5 / 37.2, 3584 42.2 / 40.0, 4096 46.8 /
// 42.2; fp32, 8192 channels: 2560 63.2 / 56.8, 4096 101.5 / 93.7.  The main
// kernel over 3 x 777 rows of 1001 in fp32, too few for that: 11.2 at 16, 12 at
// 24, 13 at 32.  Sized for vector loads: it sizes a workspace too, which must
// not depend on the current device or on strides.
//
// Packed sequences count for the rows they can have.  Their workgroups' sums
// are numbered through the pieces that the sequences are cut into where that
// bounds them lower than B times the longest sequence (14336 channels: 64
// sequences in 65536 rows, T not stated, 165 MB of sums instead of 9.4 GB;
// seven prompts in 6000 rows, 156 us instead of 161, T not stated 196).
void conv_bwd_plan(int64_t B, int64_t T, int64_t rows, int64_t C, ConvArgs* a) {
  const int64_t all = B * T < rows ? B * T : rows;
  int64_t steps = (C + 255) / 256 * all / 32 >= 2048 ? 32 : kConvTile;
  // the grid's x dimension holds (tiles / 4) x (channel blocks, at most one
  // per 64 channels)
  while (conv_groups(T, steps) * ((C + 63) / 64) > kMaxGrid) steps *= 2;
  a->steps = (int)steps;
  int64_t pieces = rows / (4 * steps) + B;
  if (pieces > rows) pieces = rows < 1 ? 1 : rows;
  a->parts = B * conv_groups(T, steps);
  a->packed = pieces < a->parts;
  if (a->packed) a->parts = pieces;
}

hipError_t launch_conv_fwd(const ConvArgs& a, bool is_bf16, hipStream_t s) {
  return is_bf16 ? launch_k<bf16, false>(a, s) : launch_k<float, false>(a, s);
}
hipError_t launch_conv_bwd(const ConvArgs& a, bool is_bf16, hipStream_t s) {
  return is_bf16 ? launch_k<bf16, true>(a, s) : launch_k<float, true>(a, s);
}

}  // namespace gdr
