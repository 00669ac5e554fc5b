// Launch interface and shared device helpers of the layer operators beside
// the gated delta rule: the short causal convolution, the selective state
// space scan and the group norm (include/gdr.h states their formulas).
#pragma once

#include "gdr_device.h"
#include "gdr_internal.h"

namespace gdr {

// The element types of activations and of weights (gdr_dtype) travel as
// "is bf16" flags.
struct ConvArgs {
  int B, T, C, K;
  int64_t rows, x_stride;
  int act;            // 1: SiLU
  int w_bf16;         // weight, bias and their gradients
  const int32_t* spans;  // [B][2] or null
  const void* x;
  const void* w;      // [C][K]
  const void* bias;   // [C] or null
  const void* state;  // [B][K-1][C] or null (zeros)
  void* y;
  void* state_out;    // or null
  // backward
  const void* dy;
  const void* dstate_out;  // or null
  void* dx;
  void* dw;
  void* dbias;        // or null
  void* dstate;       // or null
  int steps;          // of one wave
  int64_t parts;      // partial sums
  int packed;         // numbered through the sequences' pieces (pieces_before)
  float* part;        // [parts][K+1][C]
};
// Fewest steps of a tile, in either direction: a sequence of no more is
// marched through by one thread per channel, which reads a row before it
// writes the output over it.
constexpr int kConvTile = 16;
// The backward's steps, parts and packed for a's B, T, rows and C.
void conv_bwd_plan(int64_t B, int64_t T, int64_t rows, int64_t C, ConvArgs* a);
hipError_t launch_conv_fwd(const ConvArgs& a, bool bf16, hipStream_t s);
hipError_t launch_conv_bwd(const ConvArgs& a, bool bf16, hipStream_t s);

struct NormArgs {
  int64_t rows, x_stride, z_stride;
  int C, G, D;        // D = C / G
  int act, center, shared;
  int w_bf16;
  float eps;
  const void* x;
  const void* w;      // [C], or [D] (shared); null: ones
  const void* bias;   // as w; null: zeros
  const void* z;      // gate or null
  void* y;
  float* stats;       // [rows][G][2]: mean, 1/sqrt(var + eps); may be null
  // backward
  const void* dy;
  void* dx;
  void* dw;
  void* dbias;
  void* dz;
  float* part;        // [parts][2][period][D]
};
struct NormPlan {
  int lanes, nv;      // lanes and vectors per lane of one group
  bool vec;
  int64_t period;     // groups after which a lane meets the same channels again
  int64_t slabs;      // waves (blocks, for lanes > 64) that cover one period
  int64_t parts;      // workgroups per slab
};
bool norm_plan(int64_t rows, int64_t C, int64_t G, int64_t xs, int64_t zs, bool bf16, NormPlan* p);
hipError_t launch_norm_fwd(const NormArgs& a, const NormPlan& p, bool bf16, hipStream_t s);
hipError_t launch_norm_bwd(const NormArgs& a, const NormPlan& p, bool bf16, hipStream_t s);

struct ScanArgs {
  int B, T, C, N, G;
  int64_t rows, u_stride, dt_stride, z_stride, b_stride, c_stride;
  int softplus;
  const int32_t* spans;
  const void* u;
  const void* dt;
  const float* A;       // [C][N]
  const void* Bm;       // [rows][G][N]
  const void* Cm;
  const float* D;       // [C] or null
  const void* z;        // or null
  const float* dt_bias; // [C] or null
  const float* S0;      // [B][C][N] or null
  void* y;
  float* S_T;           // or null
  float* ckpt;          // [slots][C][Np]: the state every few steps, or null
  // chunked form (chunks > 1): the state (or adjoint) before every chunk and
  // the summed steps of every chunk
  int chunk;            // steps, a multiple of the tile
  int chunks;           // of the longest sequence
  float* edge;          // [slots][C][Np]
  float* dsum;          // [slots][C]
  // backward
  const void* dy;
  const float* dS_T;    // or null
  void* du;
  void* ddt;
  float* dA;
  void* dB;
  void* dC;
  float* dD;
  void* dz;
  float* ddt_bias;
  float* dS0;           // or null
  int64_t parts;        // partial sums
  int packed;           // numbered through the sequences' chunks (pieces_before)
  float* pA;            // [parts]: partial dA [C][Np], dD [C], ddt_bias [C]
  float* pB;            // [2][channel tiles][rows][G][N] partial dB, dC
};
// Padded states per channel, steps between saved states, channels of one
// workgroup.
int scan_padded(int64_t N);
int scan_save_steps(int64_t N);
int scan_channels();
// Steps of one chunk, a multiple of 16, from a's B, T, C, N, G and rows;
// stride: the widest row in elements.
int64_t scan_chunk(const ScanArgs& a, int64_t stride, bool bwd);
hipError_t launch_scan_fwd(const ScanArgs& a, bool bf16, hipStream_t s);
hipError_t launch_scan_bwd(const ScanArgs& a, bool bf16, hipStream_t s);

// Workgroups of 256 along a grid's x dimension, whose threads have to stay
// below 2^32.
constexpr int64_t kMaxGrid = (INT64_C(1) << 24) - 1;

// ---- device helpers ---------------------------------------------------------

// Rows of sequence b, held inside [0, rows) and to T steps whatever spans
// holds.
struct Span {
  int64_t first;
  int len;
};
__device__ __forceinline__ Span span_of(const int32_t* spans, int b, int T, int64_t rows) {
  if (spans == nullptr) return Span{(int64_t)b * T, T};
  int64_t s = spans[2 * b], e = spans[2 * b + 1];
  s = s < 0 ? 0 : (s > rows ? rows : s);
  e = e > rows ? rows : e;
  int64_t n = e - s;
  n = n < 0 ? 0 : (n > T ? T : n);
  return Span{s, (int)n};
}

// Pieces of n steps that the sequences before b are cut into, summed by the
// 64 lanes of a wave.  Disjoint sequences have at most rows / n + B pieces,
// and at most one a row.
__device__ __forceinline__ int64_t pieces_before(const int32_t* spans, int b, int T, int64_t rows,
                                                 int n) {
  int64_t s = 0;
  for (int i = threadIdx.x & 63; i < b; i += 64)
    s += ((int64_t)span_of(spans, i, T, rows).len + n - 1) / n;
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) s += __shfl_xor((long long)s, m, 64);
  return s;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// 1 / (1 + e^-x): the exponential overflows to inf for x < -88, whose
// reciprocal is the 0 that is meant.
__device__ __forceinline__ float sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.f + exp2_hw(-kLog2e * x));
}

// act(x), and its derivative
__device__ __forceinline__ float silu(float x) { return x * sigmoid(x); }
__device__ __forceinline__ float dsilu(float x, float sg) { return sg * (1.f + x * (1.f - sg)); }

// log(1 + e^x) = max(x, 0) + log1p(t), t = e^-|x| in (0, 1].  With w = 1 + t
// as rounded, log1p(t) = log(w + c) for c = t - (w - 1), formed exactly, of
// which log(w) + c leaves c t / w: below 1.5 2^-24 of log1p(t) for any t, so
// that small steps (t down to the smallest float, where w = 1) keep their
// relative accuracy.
__device__ __forceinline__ float softplus(float x) {
  const float t = exp2_hw(-kLog2e * fabsf(x));
  const float w = 1.f + t;
  return fmaxf(x, 0.f) + fmaf(kLn2, __builtin_amdgcn_logf(w), t - (w - 1.f));
}

// a + b with their upper halves (32 lanes) or odd rows (16 lanes) swapped for
// the other's lower or even ones: lanes of the lower half (even rows) get the
// sum of a's two halves (rows), the others that of b's.  With a = b: every
// lane the sum over both.
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

// V consecutive elements: one, or a vector of 8 or 16 bytes.
template <typename T, int V>
struct Pack {
  T v[V];
};
template <>
struct Pack<float, 4> {
  float4 v;
};
template <>
struct Pack<bf16, 8> {
  uint4 v;
};
template <>
struct Pack<bf16, 4> {
  uint2 v;
};
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load_pack(const T* p) {
  Pack<T, V> r;
  if constexpr (V == 1) {
    r.v[0] = *p;
  } else {
    r = *reinterpret_cast<const Pack<T, V>*>(p);
  }
  return r;
}
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> zero_pack() {
  Pack<T, V> r;
  __builtin_memset(&r, 0, sizeof(r));
  return r;
}
__device__ __forceinline__ void unpack(const Pack<float, 1>& p, float (&f)[1]) { f[0] = p.v[0]; }
__device__ __forceinline__ void unpack(const Pack<bf16, 1>& p, float (&f)[1]) {
  f[0] = to_f32(p.v[0]);
}
__device__ __forceinline__ void unpack(const Pack<float, 4>& p, float (&f)[4]) {
  f[0] = p.v.x;
  f[1] = p.v.y;
  f[2] = p.v.z;
  f[3] = p.v.w;
}
__device__ __forceinline__ void unpack(const Pack<bf16, 8>& p, float (&f)[8]) {
  const uint32_t w[4] = {p.v.x, p.v.y, p.v.z, p.v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack(const Pack<bf16, 4>& p, float (&f)[4]) {
  f[0] = __uint_as_float(p.v.x << 16);
  f[1] = __uint_as_float(p.v.x & 0xffff0000u);
  f[2] = __uint_as_float(p.v.y << 16);
  f[3] = __uint_as_float(p.v.y & 0xffff0000u);
}
// V floats, each rounded to nearest even.
__device__ __forceinline__ void pack(const float (&f)[1], Pack<float, 1>& p) { p.v[0] = f[0]; }
__device__ __forceinline__ void pack(const float (&f)[1], Pack<bf16, 1>& p) {
  p.v[0].bits = static_cast<uint16_t>(cvt_pk_bf16(f[0], f[0]));
}
__device__ __forceinline__ void pack(const float (&f)[4], Pack<float, 4>& p) {
  p.v = float4{f[0], f[1], f[2], f[3]};
}
__device__ __forceinline__ void pack(const float (&f)[4], Pack<bf16, 4>& p) {
  p.v = uint2{cvt_pk_bf16(f[0], f[1]), cvt_pk_bf16(f[2], f[3])};
}
__device__ __forceinline__ void pack(const float (&f)[8], Pack<bf16, 8>& p) {
  p.v = uint4{cvt_pk_bf16(f[0], f[1]), cvt_pk_bf16(f[2], f[3]), cvt_pk_bf16(f[4], f[5]),
              cvt_pk_bf16(f[6], f[7])};
}
template <typename T, int V>
__device__ __forceinline__ void store_pack(T* p, const float (&f)[V]) {
  Pack<T, V> x;
  pack(f, x);
  *reinterpret_cast<Pack<T, V>*>(p) = x;
}

// A buffer resource: a base that the whole wave shares, 32 bits of offset per
// lane, and a bound past which loads give zero and stores are dropped.  An
// absent tensor is a buffer of no bytes, read without a branch.
struct Buffer {
  const char* p;
  uint32_t bytes;
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t resource() const {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(p), 0, (int)bytes, 0x00020000);
  }
};
__device__ __forceinline__ Buffer buffer_of(const void* p, int64_t offset, int64_t bytes) {
  return Buffer{static_cast<const char*>(p) + offset, (uint32_t)bytes};
}
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> get_pack(Buffer b, uint32_t offset) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  constexpr int kBytes = V * sizeof(T);
  if constexpr (kBytes == 2)
    return __builtin_bit_cast(
        Pack<T, V>, __builtin_amdgcn_raw_buffer_load_b16(b.resource(), (int)offset, 0, 0));
  else if constexpr (kBytes == 4)
    return __builtin_bit_cast(
        Pack<T, V>, __builtin_amdgcn_raw_buffer_load_b32(b.resource(), (int)offset, 0, 0));
  else if constexpr (kBytes == 8)
    return __builtin_bit_cast(
        Pack<T, V>,
        (u32x2)__builtin_amdgcn_raw_buffer_load_b64(b.resource(), (int)offset, 0, 0));
  else
    return __builtin_bit_cast(
        Pack<T, V>,
        (u32x4)__builtin_amdgcn_raw_buffer_load_b128(b.resource(), (int)offset, 0, 0));
}

// N consecutive weights of either type from element `first` of a tensor of
// `count`, loaded raw without a branch (what the type does not ask for lies
// past the end and costs no memory; a null tensor gives zeros) and converted
// at use.  VEC: `first` and N are multiples of four.
template <int N, bool VEC>
struct Weights {
  static constexpr uint32_t kPastEnd = 0xf0000000u;  // weights end below 2^26
  static constexpr int kUnit = VEC ? (N % 8 == 0 ? 8 : 4) : 1;
  static constexpr int kUnits = N / kUnit;
  Pack<bf16, kUnit> lo[kUnits];         // the bf16 ones, or the first four floats of eight
  Pack<float, VEC ? 4 : 1> hi[kUnits];  // the floats, or the last four of eight

  __device__ __forceinline__ void load(const void* p, int64_t first, int64_t count, int is_bf16) {
    const uint32_t size = is_bf16 ? 2 : 4;
    const Buffer b = buffer_of(p, 0, p != nullptr ? count * size : 0);
    const uint32_t at = (uint32_t)first * size;
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      const uint32_t o = at + size * kUnit * k;
      lo[k] = get_pack<bf16, kUnit>(b, kUnit == 8 || is_bf16 ? o : kPastEnd);
      hi[k] = get_pack<float, VEC ? 4 : 1>(b, is_bf16 ? kPastEnd : o + (kUnit == 8 ? 16 : 0));
    }
  }
  __device__ __forceinline__ void get(int is_bf16, float (&w)[N]) const {
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      float f[kUnit], g[VEC ? 4 : 1];
      unpack(lo[k], f);
      unpack(hi[k], g);
      if constexpr (kUnit == 8) {
        const float4 first = __builtin_bit_cast(float4, lo[k]);
        const float half[4] = {first.x, first.y, first.z, first.w};
#pragma unroll
        for (int e = 0; e < 8; ++e)
          w[8 * k + e] = is_bf16 ? f[e] : (e < 4 ? half[e & 3] : g[e & 3]);
      } else {
#pragma unroll
        for (int e = 0; e < kUnit; ++e) w[kUnit * k + e] = is_bf16 ? f[e] : g[e];
      }
    }
  }
};
__device__ __forceinline__ void st_weight(void* p, int64_t i, float x, int is_bf16) {
  if (is_bf16)
    static_cast<bf16*>(p)[i] = from_f32<bf16>(x);
  else
    static_cast<float*>(p)[i] = x;
}

// Sums over the rows of part[rows][width] by a workgroup of 256: 16 columns,
// of which c is this thread's, and 16 row lanes, in a fixed order.  The sum
// comes out in the first 16 threads.
constexpr int kSumCols = 16;
__device__ __forceinline__ float column_sum(const float* __restrict__ part, int64_t rows,
                                            int64_t width, int64_t c) {
  __shared__ float red[16][kSumCols + 1];
  const int tc = threadIdx.x % kSumCols, tr = threadIdx.x / kSumCols;
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  if (c < width) {
    int64_t r = tr;
    for (; r + 48 < rows; r += 64)
#pragma unroll
      for (int k = 0; k < 4; ++k) s[k] += part[(r + 16 * k) * width + c];
    for (; r < rows; r += 16) s[0] += part[r * width + c];
  }
  red[tr][tc] = (s[0] + s[1]) + (s[2] + s[3]);
  __syncthreads();
  float t = red[0][tc];
  if (tr == 0)
#pragma unroll
    for (int k = 1; k < 16; ++k) t += red[k][tc];
  return t;
}
}  // namespace gdr
