// Linear attention with a decay for each head on gfx950:
//   S_t = g_t S_{t-1} + v_t k_t^T,  y_t = scale S_t q_t,  g_t = exp(log_g_t).
// The adjoint D_t = scale dy_t q_t^T + g_{t+1} D_{t+1} gives dq = scale S^T dy,
// dk = D^T v, dv = D k: the forward's form with the roles of the tensors
// turned (and, for dk and dv, with time reversed), so one kernel serves all:
//   state[o][i] <- g state + u V[o] K[i];  out[o] = s sum_i state[o][i] Q[i]
//   y: (Q, K, V) = (q, k, v);  dq: (dy, v, k);  dk: (v, dy, q);  dv: (k, q, dy).
//
// dlog_g_t is what flows through the decay of step t: the sum of
//   A_ij = scale exp(..) (q_i k_j) (dy_i v_j) over i >= t > j,
// which is sum_{i >= t} (a_i - b_i) + <dS_T, S_T> with a_i the sum of A_ij over
// j < i (q_i times the part of dq_i that comes from earlier steps) and b_j that
// over i > j.  The term i = j, which both would hold, is left out of both, so
// that strong decays do not leave a small difference of large sums.
#include "gdr_layer.h"

namespace gdr {
namespace {

constexpr int kThreads = 256;
constexpr int kWaveRows = kLinStepRows / (kThreads / 64);

__device__ __forceinline__ float wave_sum(float x) {
  x = rowsum16(x);
  x = swap16_sum(x, x);
  return swap32_sum(x, x);
}

__device__ __forceinline__ float log_decay(const LinArgs& a, int64_t row, int h) {
  if (a.log_g == nullptr) return 0.f;
  const int64_t at = a.per_head ? h : row * a.g_stride + h;
  return a.g_bf16 ? to_f32(static_cast<const bf16*>(a.log_g)[at])
                  : static_cast<const float*>(a.log_g)[at];
}

// One of the four products (see above).
struct Role {
  const void* Q;
  const void* K;
  const void* V;
  const void* R;       // rows that out's earlier part is multiplied with, or null
  int64_t sq, sk, sv, sr;
  int dq, dk, dv, dr;  // value heads per head of each
  int Ni, No;
  float u, s;          // factors of the update and of the output
  int reverse;
  int transposed;      // the state lies [i][o]
  const float* first;  // [B][first_per][Hv] states, of which each first one, or null
  int first_per;
  float* last;         // [B][Hv] states or null
  float* save;         // [B][2][Hv] states, the first and the last, or null
  void* out;           // [rows][Hv][No], or null
  float* part;         // the same in fp32, or null
  float* flow;         // [tiles][rows][Hv]: R out, without the step's own term
};

// A step at a time: a wave holds kWaveRows rows of the state, a lane every
// 64th column.
template <typename T>
__global__ __launch_bounds__(kThreads) void lin_step_kernel(LinArgs a, Role r) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int h = blockIdx.y, b = blockIdx.z;
  const int o0 = blockIdx.x * kLinStepRows + wave * kWaveRows;
  const Span sp = span_of(a.spans, b, a.T, a.rows);
  const int64_t size = (int64_t)r.Ni * r.No;
  const float* const first =
      r.first != nullptr ? r.first + ((int64_t)b * r.first_per * a.Hv + h) * size : nullptr;
  float S[kWaveRows][4];
#pragma unroll
  for (int j = 0; j < kWaveRows; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int o = o0 + j, i = lane + 64 * e;
      S[j][e] = first != nullptr && o < r.No && i < r.Ni
                    ? first[r.transposed ? i * r.No + o : o * r.Ni + i]
                    : 0.f;
    }
  auto store = [&](float* to) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < kWaveRows; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int o = o0 + j, i = lane + 64 * e;
        if (o < r.No && i < r.Ni) to[r.transposed ? i * r.No + o : o * r.Ni + i] = S[j][e];
      }
  };
  if (r.save != nullptr) store(r.save + ((int64_t)b * 2 * a.Hv + h) * size);
  __shared__ float red[kThreads / 64];
  for (int t = 0; t < sp.len; ++t) {
    const int64_t row = sp.first + (r.reverse ? sp.len - 1 - t : t);
    const T* const Q = static_cast<const T*>(r.Q) + row * r.sq + (int64_t)(h / r.dq) * r.Ni;
    const T* const K = static_cast<const T*>(r.K) + row * r.sk + (int64_t)(h / r.dk) * r.Ni;
    const T* const V = static_cast<const T*>(r.V) + row * r.sv + (int64_t)(h / r.dv) * r.No;
    const float g = expf(log_decay(a, row, h));
    float q[4], k[4], own = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = lane + 64 * e;
      q[e] = i < r.Ni ? to_f32(Q[i]) : 0.f;
      k[e] = i < r.Ni ? to_f32(K[i]) * r.u : 0.f;
      own = fmaf(q[e], k[e], own);
    }
    own = wave_sum(own);
    float flow = 0.f;
#pragma unroll
    for (int j = 0; j < kWaveRows; ++j) {
      const int o = o0 + j;
      const bool in = o < r.No;
      const float v = in ? to_f32(V[o]) : 0.f;
      float x = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (!r.reverse) S[j][e] *= g;
        x = fmaf(S[j][e], q[e], x);
        S[j][e] = fmaf(v, k[e], S[j][e]);
        if (r.reverse) S[j][e] *= g;
      }
      x = wave_sum(x);
      if (r.flow != nullptr && in) {
        const T* const R = static_cast<const T*>(r.R) + row * r.sr + (int64_t)(h / r.dr) * r.No;
        flow = fmaf(to_f32(R[o]), r.s * x, flow);
      }
      x = r.s * fmaf(v, own, x);
      if (lane == 0 && in) {
        const int64_t at = (row * a.Hv + h) * r.No + o;
        if (r.out != nullptr) st(static_cast<T*>(r.out), at, x);
        if (r.part != nullptr) r.part[at] = x;
      }
    }
    if (r.flow != nullptr) {
      __syncthreads();
      if (lane == 0) red[wave] = flow;
      __syncthreads();
      if (threadIdx.x == 0)
        r.flow[((int64_t)blockIdx.x * a.rows + row) * a.Hv + h] =
            (red[0] + red[1]) + (red[2] + red[3]);
    }
  }
  if (r.last != nullptr) store(r.last + ((int64_t)b * a.Hv + h) * size);
  if (r.save != nullptr) store(r.save + (((int64_t)b * 2 + 1) * a.Hv + h) * size);
}

// Sums of the fp32 parts over a key head's value heads.
template <typename T>
__global__ __launch_bounds__(kThreads) void lin_heads_sum(LinArgs a) {
  const int reps = a.Hv / a.Hk, b = blockIdx.y;
  const Span sp = span_of(a.spans, b, a.T, a.rows);
  const int64_t n = (int64_t)sp.len * a.Hk * a.Dk, start = sp.first * a.Hk * a.Dk;
  const float* const part = blockIdx.z == 0 ? a.dq_part : a.dk_part;
  T* const out = static_cast<T*>(blockIdx.z == 0 ? a.dq : a.dk);
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n;
       i += (int64_t)gridDim.x * kThreads) {
    const int64_t at = start + i;
    const int d = at % a.Dk;
    const int64_t rh = at / a.Dk;  // row and key head
    const float* const p = part + (rh / a.Hk * a.Hv + rh % a.Hk * reps) * a.Dk + d;
    float s = 0.f;
    for (int j = 0; j < reps; ++j) s += p[(int64_t)j * a.Dk];
    st(out, at, s);
  }
}

// dlog_g from the flows: one wave a sequence and head walks the steps from the
// end, 64 at a time, sums in 64 bits.
__global__ __launch_bounds__(64) void lin_flow_kernel(LinArgs a, int tiles_q, int tiles_k) {
  const int h = blockIdx.x, b = blockIdx.y, lane = threadIdx.x;
  const Span sp = span_of(a.spans, b, a.T, a.rows);
  double carry = 0.0;
  if (a.dS_T != nullptr) {
    const int64_t n = (int64_t)a.Dk * a.Dv;
    const float* const d = a.dS_T + ((int64_t)b * a.Hv + h) * n;
    const float* const S = a.ckpt + (((int64_t)b * 2 + 1) * a.Hv + h) * n;
    for (int64_t i = lane; i < n; i += 64) carry += (double)d[i] * (double)S[i];
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) carry += __shfl_xor(carry, m, 64);
  }
  const float* const fa = a.flow;
  const float* const fb = a.flow + (int64_t)tiles_q * a.rows * a.Hv;
  double head = 0.0;
  for (int t0 = (sp.len - 1) & ~63; t0 >= 0; t0 -= 64) {
    const int t = t0 + lane;
    double x = 0.0;
    const int64_t row = sp.first + t;
    if (t < sp.len) {
      for (int i = 0; i < tiles_q; ++i) x += (double)fa[((int64_t)i * a.rows + row) * a.Hv + h];
      for (int i = 0; i < tiles_k; ++i) x -= (double)fb[((int64_t)i * a.rows + row) * a.Hv + h];
    }
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {  // sums over the lanes from here on
      const double y = __shfl_down(x, m, 64);
      x += lane + m < 64 ? y : 0.0;
    }
    x += carry;
    carry = __shfl(x, 0, 64);
    if (t < sp.len) {
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
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) head += __shfl_xor(head, m, 64);
  if (lane == 0) a.head_sums[(int64_t)b * a.Hv + h] = (float)head;
}

__global__ __launch_bounds__(kThreads) void lin_head_kernel(LinArgs a) {
  const int h = blockIdx.x * kThreads + threadIdx.x;
  if (h >= a.Hv) return;
  double s = 0.0;
  for (int b = 0; b < a.B; ++b) s += (double)a.head_sums[(int64_t)b * a.Hv + h];
  st_weight(a.dlog_g, h, (float)s, a.g_bf16);
}

template <typename T>
hipError_t step(const LinArgs& a, const Role& r, hipStream_t s) {
  const unsigned tiles = (r.No + kLinStepRows - 1) / kLinStepRows;
  hipLaunchKernelGGL(lin_step_kernel<T>, dim3(tiles, a.Hv, a.B), dim3(kThreads), 0, s, a, r);
  const hipError_t e = hipGetLastError();
  note_launch(s);
  return e;
}

template <typename T>
hipError_t fwd(const LinArgs& a, hipStream_t s) {
  const int reps = a.Hv / a.Hk;
  return step<T>(a, Role{a.q, a.k, a.v, nullptr, a.q_stride, a.k_stride, a.v_stride, 0, reps, reps,
                         1, 1, a.Dk, a.Dv, 1.f, a.scale, 0, 0, a.S0, 1, a.S_T, a.ckpt, a.y,
                         nullptr, nullptr},
                 s);
}

template <typename T>
hipError_t bwd(const LinArgs& a, hipStream_t s) {
  const int reps = a.Hv / a.Hk;
  const int64_t wide = (int64_t)a.Hv * a.Dv;
  const int tiles = (a.Dk + kLinStepRows - 1) / kLinStepRows;
  const bool flows = a.dlog_g != nullptr;
  Role q{a.dy, a.v, a.k, a.q, wide, a.v_stride, a.k_stride, a.q_stride, 1, 1, reps, reps, a.Dv,
         a.Dk, 1.f, a.scale, 0, 1, a.ckpt, 2, nullptr, nullptr, reps > 1 ? nullptr : a.dq, a.dq_part,
         flows ? a.flow : nullptr};
  Role k{a.v, a.dy, a.q, a.k, a.v_stride, wide, a.q_stride, a.k_stride, 1, 1, reps, reps, a.Dv,
         a.Dk, a.scale, 1.f, 1, 1, a.dS_T, 1, nullptr, nullptr, reps > 1 ? nullptr : a.dk, a.dk_part,
         flows ? a.flow + (int64_t)tiles * a.rows * a.Hv : nullptr};
  Role v{a.k, a.q, a.dy, nullptr, a.k_stride, a.q_stride, wide, 0, reps, reps, 1, 1, a.Dk, a.Dv,
         a.scale, 1.f, 1, 0, a.dS_T, 1, a.dS0, nullptr, a.dv, nullptr, nullptr};
  hipError_t e = step<T>(a, q, s);
  if (e == hipSuccess) e = step<T>(a, k, s);
  if (e == hipSuccess) e = step<T>(a, v, s);
  if (e == hipSuccess && reps > 1) {
    const int64_t blocks = ((int64_t)a.T * a.Hk * a.Dk + kThreads - 1) / kThreads;
    hipLaunchKernelGGL(lin_heads_sum<T>,
                       dim3((unsigned)(blocks < 1 ? 1 : blocks > 1024 ? 1024 : blocks), a.B, 2),
                       dim3(kThreads), 0, s, a);
    e = hipGetLastError();
    note_launch(s);
  }
  if (e == hipSuccess && flows) {
    hipLaunchKernelGGL(lin_flow_kernel, dim3(a.Hv, a.B), dim3(64), 0, s, a, tiles, tiles);
    e = hipGetLastError();
    note_launch(s);
    if (e == hipSuccess && a.per_head) {
      hipLaunchKernelGGL(lin_head_kernel, dim3((a.Hv + kThreads - 1) / kThreads), dim3(kThreads),
                         0, s, a);
      e = hipGetLastError();
      note_launch(s);
    }
  }
  return e;
}

}  // namespace

hipError_t launch_lin_fwd(const LinArgs& a, bool is_bf16, hipStream_t s) {
  return is_bf16 ? fwd<bf16>(a, s) : fwd<float>(a, s);
}
hipError_t launch_lin_bwd(const LinArgs& a, bool is_bf16, hipStream_t s) {
  return is_bf16 ? bwd<bf16>(a, s) : bwd<float>(a, s);
}

}  // namespace gdr
