// Host side of the layer operators' C ABI (include/gdr.h): argument
// validation, size queries and launches of the short causal convolution, the
// selective state space scan and the group norm.  As in gdr_api.hip, every
// check runs on the host before anything is enqueued.
#include <math.h>
#include <stdint.h>

#include "../../include/gdr.h"
#include "gdr_layer.h"

namespace {

constexpr int64_t kMaxChannels = INT64_C(1) << 20;
constexpr int64_t kMaxRows = INT32_MAX / 2;  // rows and steps; twice it still is an int
constexpr int64_t kMaxStride = INT32_MAX;
constexpr int64_t kMaxScanStride = INT64_C(1) << 25;  // 16 rows of 4 bytes in 32 bits
constexpr int64_t kMaxBatch = 65535;  // sequences index grid y, groups z
constexpr int64_t kMaxIndex = INT64_C(1) << 61;

int64_t round_up256(int64_t x) { return (x + 255) & ~int64_t(255); }

bool product_ok(int64_t a, int64_t b, int64_t* out) {
  if (a != 0 && b > kMaxIndex / a) return false;
  *out = a * b;
  return true;
}

bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

template <int N>
int pointers_ok(const void* const (&required)[N], bool needed) {
  if (needed)
    for (const void* p : required)
      if (p == nullptr) return GDR_ERR_NULL_ARG;
  return GDR_OK;
}
template <int N>
int alignment_ok(const void* const (&ptrs)[N]) {
  for (const void* p : ptrs)
    if (misaligned(p)) return GDR_ERR_ALIGNMENT;
  return GDR_OK;
}

bool dtype_ok(int32_t d) { return d == GDR_F32 || d == GDR_BF16; }
bool stride_ok(int64_t* s, int64_t width, int64_t most = kMaxStride) {
  if (*s == 0) *s = width;
  return *s >= width && *s <= most;
}

// B, T, rows of a shape with sequences
int sequences_ok(int64_t B, int64_t T, int64_t rows) {
  if (B < 0 || T < 0 || rows < 0 || B > kMaxBatch || T > kMaxRows || rows > kMaxRows)
    return GDR_ERR_BAD_DIM;
  return GDR_OK;
}

int check(const gdr_conv_shape* in, gdr_conv_shape* s) {
  if (in == nullptr) return GDR_ERR_NULL_ARG;
  *s = *in;
  const int st = sequences_ok(s->B, s->T, s->rows);
  if (st != GDR_OK) return st;
  if (s->C < 1 || s->C > kMaxChannels || s->K < 1 || s->K > GDR_CONV_MAX_TAPS)
    return GDR_ERR_BAD_DIM;
  if (!dtype_ok(s->dtype) || !dtype_ok(s->wdtype)) return GDR_ERR_BAD_DTYPE;
  if (s->act != GDR_ACT_NONE && s->act != GDR_ACT_SILU) return GDR_ERR_BAD_ACT;
  if (!stride_ok(&s->x_stride, s->C)) return GDR_ERR_BAD_STRIDE;
  return GDR_OK;
}

int check(const gdr_scan_shape* in, gdr_scan_shape* s) {
  if (in == nullptr) return GDR_ERR_NULL_ARG;
  *s = *in;
  const int st = sequences_ok(s->B, s->T, s->rows);
  if (st != GDR_OK) return st;
  if (s->C < 1 || s->C > kMaxChannels || s->N < 1 || s->N > GDR_SCAN_MAX_STATES || s->G < 1 ||
      s->G > s->C || s->G > kMaxBatch || s->C % s->G != 0)
    return GDR_ERR_BAD_DIM;
  if (!dtype_ok(s->dtype)) return GDR_ERR_BAD_DTYPE;
  if (s->softplus != 0 && s->softplus != 1) return GDR_ERR_BAD_ACT;
  const int64_t most = kMaxScanStride;
  if (!stride_ok(&s->u_stride, s->C, most) || !stride_ok(&s->dt_stride, s->C, most) ||
      !stride_ok(&s->z_stride, s->C, most) || !stride_ok(&s->b_stride, s->G * s->N, most) ||
      !stride_ok(&s->c_stride, s->G * s->N, most))
    return GDR_ERR_BAD_STRIDE;
  return GDR_OK;
}

int check(const gdr_norm_shape* in, gdr_norm_shape* s, gdr::NormPlan* p) {
  if (in == nullptr) return GDR_ERR_NULL_ARG;
  *s = *in;
  if (s->rows < 0 || s->rows > kMaxRows || s->C < 1 || s->C > kMaxChannels || s->G < 1 ||
      s->G > s->C || s->C % s->G != 0)
    return GDR_ERR_BAD_DIM;
  if (!dtype_ok(s->dtype) || !dtype_ok(s->wdtype)) return GDR_ERR_BAD_DTYPE;
  if (s->act != GDR_ACT_NONE && s->act != GDR_ACT_SILU) return GDR_ERR_BAD_ACT;
  if (!(s->eps >= 0.f) || isinf(s->eps)) return GDR_ERR_BAD_EPS;
  if (!stride_ok(&s->x_stride, s->C) || !stride_ok(&s->z_stride, s->C)) return GDR_ERR_BAD_STRIDE;
  if (s->rows * s->G > INT32_MAX) return GDR_ERR_OVERFLOW;
  if (!gdr::norm_plan(s->rows, s->C, s->G, s->x_stride, s->z_stride, s->dtype == GDR_BF16, p))
    return GDR_ERR_BAD_DIM;
  return GDR_OK;
}

// ---- scan: chunks and buffers ------------------------------------------------
struct ScanSizes {
  int64_t chunk, chunks;     // of the longest sequence
  int64_t parts;             // partial sums of the backward
  bool packed;
  int64_t edge, dsum, part, bc, bytes;  // byte offsets of the workspace, its size
  int64_t ckpt;              // bytes of the save buffer
};

int scan_sizes(const gdr_scan_shape& s, bool bwd, ScanSizes* z) {
  const int64_t np = gdr::scan_padded(s.N), tile = gdr::scan_save_steps(s.N);
  int64_t stride = s.C > s.G * s.N ? s.C : s.G * s.N;
  for (int64_t w : {s.u_stride, s.dt_stride, s.z_stride, s.b_stride, s.c_stride})
    if (w > stride) stride = w;
  gdr::ScanArgs a{};
  a.B = (int)s.B;
  a.T = (int)s.T;
  a.C = (int)s.C;
  a.N = (int)s.N;
  a.G = (int)s.G;
  a.rows = s.rows;
  z->chunk = gdr::scan_chunk(a, stride, bwd);
  z->chunks = s.T > 0 ? (s.T + z->chunk - 1) / z->chunk : 1;
  const int64_t tiles = (s.C / s.G + gdr::scan_channels() - 1) / gdr::scan_channels();
  if (s.G * tiles * z->chunks > gdr::kMaxGrid) return GDR_ERR_OVERFLOW;
  int64_t state, x;
  if (!product_ok(s.C, np * 4, &state) || !product_ok(state, s.rows / tile + s.B + 1, &z->ckpt))
    return GDR_ERR_OVERFLOW;
  z->edge = 0;
  z->dsum = 0;
  z->bytes = 0;
  if (z->chunks > 1) {
    const int64_t slots = s.rows / z->chunk + s.B + 1;
    if (!product_ok(state, slots, &x)) return GDR_ERR_OVERFLOW;
    z->dsum = round_up256(x);
    z->bytes = z->dsum + round_up256(slots * s.C * 4);
  }
  if (bwd) {
    // one for every chunk that the rows can have, where those are fewer than
    // B times the longest sequence's (4096 channels of 16 states: 1000
    // sequences in 65536 rows, T not stated, 300 MB instead of 4.7 GB)
    int64_t pieces = s.rows / z->chunk + s.B;
    if (pieces > s.rows) pieces = s.rows < 1 ? 1 : s.rows;
    z->parts = s.B * z->chunks;
    z->packed = pieces < z->parts;
    if (z->packed) z->parts = pieces;
    z->part = z->bytes;
    if (!product_ok(s.C * (np + 2) * 4, z->parts, &x)) return GDR_ERR_OVERFLOW;
    z->bytes += round_up256(x);
    z->bc = z->bytes;
    if (!product_ok(s.rows * 8, s.G * s.N * tiles, &x)) return GDR_ERR_OVERFLOW;
    z->bytes += round_up256(x);
  }
  return GDR_OK;
}

gdr::ScanArgs scan_args(const gdr_scan_shape& s, const ScanSizes& z, const void* u, const void* dt,
                        const float* A, const void* Bm, const void* Cm, const float* D,
                        const void* zg, const float* dt_bias, const int32_t* spans, void* ws) {
  gdr::ScanArgs a{};
  a.B = (int)s.B;
  a.T = (int)s.T;
  a.C = (int)s.C;
  a.N = (int)s.N;
  a.G = (int)s.G;
  a.rows = s.rows;
  a.u_stride = s.u_stride;
  a.dt_stride = s.dt_stride;
  a.z_stride = s.z_stride;
  a.b_stride = s.b_stride;
  a.c_stride = s.c_stride;
  a.softplus = s.softplus;
  a.spans = spans;
  a.u = u;
  a.dt = dt;
  a.A = A;
  a.Bm = Bm;
  a.Cm = Cm;
  a.D = D;
  a.z = zg;
  a.dt_bias = dt_bias;
  a.chunk = (int)z.chunk;
  a.chunks = (int)z.chunks;
  char* const w = static_cast<char*>(ws);
  if (z.chunks > 1) {
    a.edge = reinterpret_cast<float*>(w + z.edge);
    a.dsum = reinterpret_cast<float*>(w + z.dsum);
  }
  return a;
}

int hip_status(hipError_t e) { return e == hipSuccess ? GDR_OK : GDR_ERR_HIP; }

// ---- the entry points' work --------------------------------------------------
gdr::ConvArgs conv_args(const gdr_conv_shape& s, const void* x, const void* w, const void* bias,
                        const void* state, const int32_t* spans) {
  gdr::ConvArgs a{};
  a.B = (int)s.B;
  a.T = (int)s.T;
  a.C = (int)s.C;
  a.K = (int)s.K;
  a.rows = s.rows;
  a.x_stride = s.x_stride;
  a.act = s.act;
  a.w_bf16 = s.wdtype == GDR_BF16;
  a.spans = spans;
  a.x = x;
  a.w = w;
  a.bias = bias;
  a.state = state;
  return a;
}

// Dense batches own exactly B T rows.
int rows_ok(int64_t B, int64_t T, int64_t rows, const int32_t* spans) {
  return spans == nullptr && rows != B * T ? GDR_ERR_BAD_DIM : GDR_OK;
}

// The rows [rows][C] of q, `stride` elements apart, against the dense output
// rows at p: apart, or the same ones of sequences that are one tile each.
static_assert(gdr::kConvTile == GDR_CONV_IN_PLACE_STEPS, "what the header promises");
int over_rows_ok(const gdr_conv_shape& s, const void* q, int64_t stride, const void* p) {
  const uintptr_t size = s.dtype == GDR_BF16 ? 2 : 4, width = s.C * size, step = stride * size;
  const uintptr_t in = reinterpret_cast<uintptr_t>(q), out = reinterpret_cast<uintptr_t>(p);
  const uintptr_t bytes = s.rows * width;
  if (out + bytes <= in || out >= in + (s.rows - 1) * step + width) return GDR_OK;
  if (out == in && stride == s.C && s.T <= GDR_CONV_IN_PLACE_STEPS) return GDR_OK;
  // (between two rows of q)
  if (out > in && (out - in) % step >= width && (out - in) % step + bytes <= step) return GDR_OK;
  return GDR_ERR_OVERLAP;
}

int conv_forward(const gdr_conv_shape* shape, const void* x, const void* w, const void* bias,
                 const void* state, const int32_t* spans, void* y, void* state_out,
                 void* stream) {
  gdr_conv_shape s;
  int st = check(shape, &s);
  if (st == GDR_OK) st = rows_ok(s.B, s.T, s.rows, spans);
  const bool has_rows = s.B > 0 && s.T > 0 && s.rows > 0;
  if (st == GDR_OK) st = pointers_ok({x, w, static_cast<const void*>(y)}, has_rows);
  if (st == GDR_OK) st = alignment_ok({x, w, bias, state, spans, y, state_out});
  if (st == GDR_OK && has_rows) st = over_rows_ok(s, x, s.x_stride, y);
  if (st != GDR_OK) return st;
  if (s.B == 0 || (!has_rows && (state_out == nullptr || s.K == 1))) return GDR_OK;
  if (w == nullptr) return GDR_ERR_NULL_ARG;
  gdr::ConvArgs a = conv_args(s, x, w, bias, state, spans);
  if (!has_rows) a.T = 0;
  a.y = y;
  a.state_out = s.K > 1 ? state_out : nullptr;
  return hip_status(gdr::launch_conv_fwd(a, s.dtype == GDR_BF16, static_cast<hipStream_t>(stream)));
}

int conv_backward_sizes(const gdr_conv_shape* shape, gdr_conv_shape* s, gdr::ConvArgs* plan,
                        int64_t* bytes) {
  const int st = check(shape, s);
  if (st != GDR_OK) return st;
  gdr::conv_bwd_plan(s->B, s->T, s->rows, s->C, plan);
  if (!product_ok(plan->parts, (s->K + 1) * s->C * 4, bytes)) return GDR_ERR_OVERFLOW;
  return GDR_OK;
}

int conv_backward(const gdr_conv_shape* shape, const void* x, const void* w, const void* bias,
                  const void* state, const int32_t* spans, const void* dy, const void* dstate_out,
                  void* dx, void* dw, void* dbias, void* dstate, void* workspace,
                  size_t workspace_bytes, void* stream) {
  gdr_conv_shape s;
  gdr::ConvArgs plan{};
  int64_t need = 0;
  int st = conv_backward_sizes(shape, &s, &plan, &need);
  if (st == GDR_OK) st = rows_ok(s.B, s.T, s.rows, spans);
  const bool has_rows = s.B > 0 && s.T > 0 && s.rows > 0;
  if (st == GDR_OK)
    st = pointers_ok({w, static_cast<const void*>(dw), static_cast<const void*>(workspace)},
                     s.B > 0);
  if (st == GDR_OK) st = pointers_ok({x, dy, static_cast<const void*>(dx)}, has_rows);
  if (st == GDR_OK)
    st = alignment_ok({x, w, bias, state, spans, dy, dstate_out, dx, dw, dbias, dstate,
                       static_cast<const void*>(workspace)});
  if (st == GDR_OK && has_rows) st = over_rows_ok(s, x, s.x_stride, dx);
  if (st == GDR_OK && has_rows) st = over_rows_ok(s, dy, s.C, dx);
  if (st != GDR_OK) return st;
  if (s.B == 0) return GDR_OK;
  if (workspace_bytes < (size_t)need) return GDR_ERR_WORKSPACE;
  gdr::ConvArgs a = conv_args(s, x, w, bias, state, spans);
  if (!has_rows) a.rows = 0;
  a.steps = plan.steps;
  a.parts = plan.parts;
  a.packed = plan.packed;
  a.dy = dy;
  a.dstate_out = s.K > 1 ? dstate_out : nullptr;
  a.dx = dx;
  a.dw = dw;
  a.dbias = dbias;
  a.dstate = s.K > 1 ? dstate : nullptr;
  a.part = static_cast<float*>(workspace);
  return hip_status(gdr::launch_conv_bwd(a, s.dtype == GDR_BF16, static_cast<hipStream_t>(stream)));
}

int scan_forward(const gdr_scan_shape* shape, const void* u, const void* dt, const float* A,
                 const void* Bm, const void* Cm, const float* D, const void* z,
                 const float* dt_bias, const float* S0, const int32_t* spans, void* y, float* S_T,
                 void* ckpt, void* workspace, size_t workspace_bytes, void* stream) {
  gdr_scan_shape s;
  ScanSizes sz;
  int st = check(shape, &s);
  if (st == GDR_OK) st = rows_ok(s.B, s.T, s.rows, spans);
  if (st == GDR_OK) st = scan_sizes(s, false, &sz);
  const bool has_rows = s.B > 0 && s.T > 0 && s.rows > 0;
  if (st == GDR_OK)
    st = pointers_ok({u, dt, static_cast<const void*>(A), Bm, Cm, static_cast<const void*>(y)},
                     has_rows);
  if (st == GDR_OK)
    st = alignment_ok({u, dt, A, Bm, Cm, D, z, dt_bias, S0, spans, y, S_T, ckpt,
                       static_cast<const void*>(workspace)});
  if (st != GDR_OK) return st;
  if (s.B == 0 || (!has_rows && S_T == nullptr)) return GDR_OK;
  if (sz.bytes > 0 && (workspace == nullptr || workspace_bytes < (size_t)sz.bytes))
    return GDR_ERR_WORKSPACE;
  if (A == nullptr) return GDR_ERR_NULL_ARG;
  gdr::ScanArgs a = scan_args(s, sz, u, dt, A, Bm, Cm, D, z, dt_bias, spans, workspace);
  if (!has_rows) a.rows = 0, a.T = 0;
  a.S0 = S0;
  a.y = y;
  a.S_T = S_T;
  a.ckpt = static_cast<float*>(ckpt);
  return hip_status(gdr::launch_scan_fwd(a, s.dtype == GDR_BF16, static_cast<hipStream_t>(stream)));
}

int scan_backward(const gdr_scan_shape* shape, const void* u, const void* dt, const float* A,
                  const void* Bm, const void* Cm, const float* D, const void* z,
                  const float* dt_bias, const int32_t* spans, const void* ckpt, const void* dy,
                  const float* dS_T, void* du, void* ddt, float* dA, void* dB, void* dC, float* dD,
                  void* dz, float* ddt_bias, float* dS0, void* workspace, size_t workspace_bytes,
                  void* stream) {
  gdr_scan_shape s;
  ScanSizes sz;
  int st = check(shape, &s);
  if (st == GDR_OK) st = rows_ok(s.B, s.T, s.rows, spans);
  if (st == GDR_OK) st = scan_sizes(s, true, &sz);
  const bool has_rows = s.B > 0 && s.T > 0 && s.rows > 0;
  if (st == GDR_OK)
    st = pointers_ok({static_cast<const void*>(A), static_cast<const void*>(dA),
                      static_cast<const void*>(workspace)},
                     s.B > 0);
  if (st == GDR_OK)
    st = pointers_ok({u, dt, Bm, Cm, ckpt, dy, static_cast<const void*>(du),
                      static_cast<const void*>(ddt), static_cast<const void*>(dB),
                      static_cast<const void*>(dC)},
                     has_rows);
  if (st == GDR_OK && has_rows && z != nullptr && dz == nullptr) st = GDR_ERR_NULL_ARG;
  if (st == GDR_OK)
    st = alignment_ok({u, dt, A, Bm, Cm, D, z, dt_bias, spans, ckpt, dy, dS_T, du, ddt, dA, dB, dC,
                       dD, dz, ddt_bias, dS0, static_cast<const void*>(workspace)});
  if (st != GDR_OK) return st;
  if (s.B == 0) return GDR_OK;
  if (workspace_bytes < (size_t)sz.bytes) return GDR_ERR_WORKSPACE;
  gdr::ScanArgs a = scan_args(s, sz, u, dt, A, Bm, Cm, D, z, dt_bias, spans, workspace);
  if (!has_rows) a.rows = 0, a.T = 0;
  a.ckpt = static_cast<float*>(const_cast<void*>(ckpt));
  a.dy = dy;
  a.dS_T = dS_T;
  a.du = du;
  a.ddt = ddt;
  a.dA = dA;
  a.dB = dB;
  a.dC = dC;
  a.dD = dD;
  a.dz = dz;
  a.ddt_bias = ddt_bias;
  a.dS0 = dS0;
  a.parts = sz.parts;
  a.packed = sz.packed;
  char* const w = static_cast<char*>(workspace);
  a.pA = reinterpret_cast<float*>(w + sz.part);
  a.pB = reinterpret_cast<float*>(w + sz.bc);
  return hip_status(gdr::launch_scan_bwd(a, s.dtype == GDR_BF16, static_cast<hipStream_t>(stream)));
}

gdr::NormArgs norm_args(const gdr_norm_shape& s, const void* x, const void* w, const void* bias,
                        const void* z) {
  gdr::NormArgs a{};
  a.rows = s.rows;
  a.x_stride = s.x_stride;
  a.z_stride = s.z_stride;
  a.C = (int)s.C;
  a.G = (int)s.G;
  a.D = (int)(s.C / s.G);
  a.act = s.act;
  a.center = s.center != 0;
  a.shared = s.shared_weight != 0;
  a.w_bf16 = s.wdtype == GDR_BF16;
  a.eps = s.eps;
  a.x = x;
  a.w = w;
  a.bias = bias;
  a.z = z;
  return a;
}

int norm_forward(const gdr_norm_shape* shape, const void* x, const void* w, const void* bias,
                 const void* z, void* y, float* stats, void* stream) {
  gdr_norm_shape s;
  gdr::NormPlan p;
  int st = check(shape, &s, &p);
  if (st == GDR_OK) st = pointers_ok({x, static_cast<const void*>(y)}, s.rows > 0);
  if (st == GDR_OK) st = alignment_ok({x, w, bias, z, y, static_cast<const void*>(stats)});
  if (st != GDR_OK || s.rows == 0) return st;
  gdr::NormArgs a = norm_args(s, x, w, bias, z);
  a.y = y;
  a.stats = stats;
  return hip_status(gdr::launch_norm_fwd(a, p, s.dtype == GDR_BF16,
                                         static_cast<hipStream_t>(stream)));
}

int64_t norm_workspace(const gdr_norm_shape& s, const gdr::NormPlan& p) {
  const int64_t D = s.C / s.G;
  // part[parts][2][period][D], or part[parts x slabs][2][D] for a shared weight
  return p.parts * 2 * (s.shared_weight != 0 ? p.slabs * D : p.period * D) * 4;
}

int norm_backward(const gdr_norm_shape* shape, const void* x, const void* w, const void* bias,
                  const void* z, const float* stats, const void* dy, void* dx, void* dw,
                  void* dbias, void* dz, void* workspace, size_t workspace_bytes, void* stream) {
  gdr_norm_shape s;
  gdr::NormPlan p;
  int st = check(shape, &s, &p);
  if (st == GDR_OK)
    st = pointers_ok({x, static_cast<const void*>(stats), dy, static_cast<const void*>(dx)},
                     s.rows > 0);
  if (st == GDR_OK && s.rows > 0 && z != nullptr && dz == nullptr) st = GDR_ERR_NULL_ARG;
  if (st == GDR_OK)
    st = alignment_ok({x, w, bias, z, stats, dy, dx, dw, dbias, dz,
                       static_cast<const void*>(workspace)});
  if (st != GDR_OK) return st;
  const bool sums = dw != nullptr || dbias != nullptr;
  if (s.rows == 0 && !sums) return GDR_OK;
  if (sums &&
      (workspace == nullptr || workspace_bytes < (size_t)norm_workspace(s, p)))
    return GDR_ERR_WORKSPACE;
  gdr::NormArgs a = norm_args(s, x, w, bias, z);
  a.stats = const_cast<float*>(stats);
  a.dy = dy;
  a.dx = dx;
  a.dw = dw;
  a.dbias = dbias;
  a.dz = dz;
  a.part = static_cast<float*>(workspace);
  return hip_status(gdr::launch_norm_bwd(a, p, s.dtype == GDR_BF16,
                                         static_cast<hipStream_t>(stream)));
}

int store_size(int st, int64_t bytes, size_t* out) {
  if (st != GDR_OK) return st;
  if (out == nullptr) return GDR_ERR_NULL_ARG;
  *out = static_cast<size_t>(bytes);
  return GDR_OK;
}

}  // namespace

extern "C" {

int gdr_conv_forward(const gdr_conv_shape* shape, const void* x, const void* weight,
                     const void* bias, const void* state, const int32_t* spans, void* y,
                     void* state_out, void* stream) {
  gdr::begin_call();
  return gdr::finish_call(
      conv_forward(shape, x, weight, bias, state, spans, y, state_out, stream), stream);
}

int gdr_conv_backward_workspace_bytes(const gdr_conv_shape* shape, size_t* out) {
  gdr_conv_shape s;
  gdr::ConvArgs plan{};
  int64_t bytes = 0;
  const int st = conv_backward_sizes(shape, &s, &plan, &bytes);
  return store_size(st, bytes, out);
}

int gdr_conv_backward(const gdr_conv_shape* shape, const void* x, const void* weight,
                      const void* bias, const void* state, const int32_t* spans, const void* dy,
                      const void* dstate_out, void* dx, void* dweight, void* dbias, void* dstate,
                      void* workspace, size_t workspace_bytes, void* stream) {
  gdr::begin_call();
  return gdr::finish_call(
      conv_backward(shape, x, weight, bias, state, spans, dy, dstate_out, dx, dweight, dbias,
                    dstate, workspace, workspace_bytes, stream),
      stream);
}

int gdr_scan_checkpoint_bytes(const gdr_scan_shape* shape, size_t* out) {
  gdr_scan_shape s;
  ScanSizes z{};
  int st = check(shape, &s);
  if (st == GDR_OK) st = scan_sizes(s, false, &z);
  return store_size(st, z.ckpt, out);
}

int gdr_scan_forward_workspace_bytes(const gdr_scan_shape* shape, size_t* out) {
  gdr_scan_shape s;
  ScanSizes z{};
  int st = check(shape, &s);
  if (st == GDR_OK) st = scan_sizes(s, false, &z);
  return store_size(st, z.bytes, out);
}

int gdr_scan_backward_workspace_bytes(const gdr_scan_shape* shape, size_t* out) {
  gdr_scan_shape s;
  ScanSizes z{};
  int st = check(shape, &s);
  if (st == GDR_OK) st = scan_sizes(s, true, &z);
  return store_size(st, z.bytes, out);
}

int gdr_scan_forward(const gdr_scan_shape* shape, const void* u, const void* dt, const float* A,
                     const void* Bm, const void* Cm, const float* D, const void* z,
                     const float* dt_bias, const float* S0, const int32_t* spans, void* y,
                     float* S_T, void* ckpt, void* workspace, size_t workspace_bytes,
                     void* stream) {
  gdr::begin_call();
  return gdr::finish_call(scan_forward(shape, u, dt, A, Bm, Cm, D, z, dt_bias, S0, spans, y, S_T,
                                       ckpt, workspace, workspace_bytes, stream),
                          stream);
}

int gdr_scan_backward(const gdr_scan_shape* shape, const void* u, const void* dt, const float* A,
                      const void* Bm, const void* Cm, const float* D, const void* z,
                      const float* dt_bias, const int32_t* spans, const void* ckpt, const void* dy,
                      const float* dS_T, void* du, void* ddt, float* dA, void* dB, void* dC,
                      float* dD, void* dz, float* ddt_bias, float* dS0, void* workspace,
                      size_t workspace_bytes, void* stream) {
  gdr::begin_call();
  return gdr::finish_call(
      scan_backward(shape, u, dt, A, Bm, Cm, D, z, dt_bias, spans, ckpt, dy, dS_T, du, ddt, dA, dB,
                    dC, dD, dz, ddt_bias, dS0, workspace, workspace_bytes, stream),
      stream);
}

int gdr_norm_forward(const gdr_norm_shape* shape, const void* x, const void* weight,
                     const void* bias, const void* z, void* y, float* stats, void* stream) {
  gdr::begin_call();
  return gdr::finish_call(norm_forward(shape, x, weight, bias, z, y, stats, stream), stream);
}

int gdr_norm_backward_workspace_bytes(const gdr_norm_shape* shape, size_t* out) {
  gdr_norm_shape s;
  gdr::NormPlan p{};
  const int st = check(shape, &s, &p);
  return store_size(st, st == GDR_OK ? norm_workspace(s, p) : 0, out);
}

int gdr_norm_backward(const gdr_norm_shape* shape, const void* x, const void* weight,
                      const void* bias, const void* z, const float* stats, const void* dy,
                      void* dx, void* dweight, void* dbias, void* dz, void* workspace,
                      size_t workspace_bytes, void* stream) {
  gdr::begin_call();
  return gdr::finish_call(norm_backward(shape, x, weight, bias, z, stats, dy, dx, dweight, dbias,
                                        dz, workspace, workspace_bytes, stream),
                          stream);
}

}  // extern "C"
