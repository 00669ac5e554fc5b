/* Host-side checks of linear attention's and the block norms' C entry points
 * (include/gdr.h) for a sanitizer build: the size queries over many shapes, up
 * to the limits, and every argument-rejection path.  Nothing here reaches the
 * device.  Exits non-zero on the first wrong status.  Built and run by
 * tests/test_block_abi.py. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "gdr.h"

static int fails = 0;
#define EXPECT(cond)                                                        \
  do {                                                                      \
    if (!(cond)) {                                                          \
      fprintf(stderr, "%s:%d: check failed: %s\n", __FILE__, __LINE__, #cond); \
      ++fails;                                                              \
    }                                                                       \
  } while (0)

static gdr_lin_shape lin(int64_t B, int64_t T, int64_t Hk, int64_t Hv, int64_t Dk, int64_t Dv, int32_t dt) {
  gdr_lin_shape s;
  memset(&s, 0, sizeof s);
  s.B = B; s.T = T; s.rows = B * T; s.Hk = Hk; s.Hv = Hv; s.Dk = Dk; s.Dv = Dv;
  s.scale = 1.f; s.dtype = dt; s.gdtype = GDR_F32;
  return s;
}
static gdr_res_shape res(int64_t rows, int64_t C, int64_t gate_rows, int32_t dt) {
  gdr_res_shape s;
  memset(&s, 0, sizeof s);
  s.rows = rows; s.C = C; s.gate_rows = gate_rows; s.alpha = 1.f; s.eps = 1e-6f;
  s.dtype = dt; s.rdtype = dt; s.wdtype = dt; s.gdtype = dt; s.post = 1; s.pre = 1;
  return s;
}
static int lin_fwd(const gdr_lin_shape* s, const void* q, void* y, const void* ckpt, void* ws, size_t n) {
  return gdr_lin_forward(s, q, q, q, q, q, 0, y, 0, (void*)ckpt, ws, n, 0);
}
static int lin_bwd(const gdr_lin_shape* s, const void* q, const void* ckpt, void* d, void* dlg, void* ws, size_t n) {
  return gdr_lin_backward(s, q, q, q, q, 0, ckpt, q, 0, d, d, d, dlg, 0, ws, n, 0);
}
static int res_fwd(const gdr_res_shape* s, const void* x, void* y, void* h) {
  return gdr_res_forward(s, x, x, 0, 0, 0, 0, 0, y, h, 0, 0);
}
static int res_bwd(const gdr_res_shape* s, const void* x, const void* dy, const void* dh, void* dg, void* dw, void* ws,
                   size_t n) {
  return gdr_res_backward(s, x, x, dg ? x : 0, x, 0, 0, 0, x, dy, dh, (void*)x, (void*)x, dg, dw, 0, 0, 0, ws, n, 0);
}

int main(void) {
  static char buf[64] __attribute__((aligned(16)));
  void* F = buf;
  void* M = buf + 4; /* misaligned */
  size_t n = 0, m = 0;
  const int64_t Ts[] = {0, 1, 8, 9, 127, 128, 129, 300, 8192, (INT64_C(1) << 30) - 1};
  const int64_t Ds[] = {1, 7, 64, 65, 128, 192, 256};
  for (size_t i = 0; i < sizeof Ts / sizeof Ts[0]; ++i)
    for (size_t j = 0; j < sizeof Ds / sizeof Ds[0]; ++j)
      for (int dt = 0; dt < 2; ++dt) {
        for (int64_t B = 0; B <= 3; ++B)
          for (int64_t R = 1; R <= 4; R += 3) {
            if (B * Ts[i] > (INT64_C(1) << 30) - 1) continue;
            gdr_lin_shape s = lin(B, Ts[i], 2, 2 * R, Ds[j], Ds[(j + 3) % 7], dt);
            const int a = gdr_lin_checkpoint_bytes(&s, &n);
            EXPECT(a == GDR_OK || a == GDR_ERR_OVERFLOW);
            if (a == GDR_OK) EXPECT(n >= (size_t)(2 * B * 2 * R * s.Dk * s.Dv * 4));
            const int b = gdr_lin_forward_workspace_bytes(&s, &n), c = gdr_lin_backward_workspace_bytes(&s, &m);
            EXPECT(b == a && c == a);
            /* packed rows: T bounds the sequences, whatever it is */
            s.T = (INT64_C(1) << 30) - 1;
            EXPECT(gdr_lin_backward_workspace_bytes(&s, &n) == a);
          }
        for (int64_t g = 0; g <= Ts[i]; g = g == 0 ? 1 : 3 * g) {
          gdr_res_shape s = res(Ts[i], 16 * Ds[j], g, dt);
          const int st = gdr_res_backward_workspace_bytes(&s, &n);
          EXPECT(st == (g > 0 && g < Ts[i] && Ts[i] % g ? GDR_ERR_BAD_DIM : GDR_OK));
        }
      }

  gdr_lin_shape s = lin(2, 200, 2, 4, 64, 64, GDR_BF16), t;
  EXPECT(gdr_lin_checkpoint_bytes(0, &n) == GDR_ERR_NULL_ARG);
  EXPECT(gdr_lin_checkpoint_bytes(&s, 0) == GDR_ERR_NULL_ARG);
  EXPECT(gdr_lin_forward_workspace_bytes(&s, &n) == GDR_OK);
  EXPECT(gdr_lin_backward_workspace_bytes(&s, &m) == GDR_OK && m > 0);
  EXPECT(lin_fwd(0, F, F, 0, F, n) == GDR_ERR_NULL_ARG);
  EXPECT(lin_fwd(&s, 0, F, 0, F, n) == GDR_ERR_NULL_ARG);
  EXPECT(lin_fwd(&s, F, 0, 0, F, n) == GDR_ERR_NULL_ARG);
  EXPECT(lin_fwd(&s, M, F, 0, F, n) == GDR_ERR_ALIGNMENT);
  EXPECT(lin_fwd(&s, F, M, 0, F, n) == GDR_ERR_ALIGNMENT);
  EXPECT(lin_fwd(&s, F, F, M, F, n) == GDR_ERR_ALIGNMENT);
  if (n > 0) EXPECT(lin_fwd(&s, F, F, 0, F, n - 1) == GDR_ERR_WORKSPACE);
  if (n > 0) EXPECT(lin_fwd(&s, F, F, 0, 0, n) == GDR_ERR_WORKSPACE);
  EXPECT(lin_bwd(&s, F, 0, F, F, F, m) == GDR_ERR_NULL_ARG);
  EXPECT(lin_bwd(&s, F, F, 0, F, F, m) == GDR_ERR_NULL_ARG);
  EXPECT(lin_bwd(&s, F, F, F, F, F, m - 1) == GDR_ERR_WORKSPACE);
  EXPECT(lin_bwd(&s, F, F, F, F, 0, m) == GDR_ERR_WORKSPACE);
  EXPECT(lin_bwd(&s, F, F, F, M, F, m) == GDR_ERR_ALIGNMENT);
  EXPECT(gdr_lin_backward(&s, F, F, F, 0, 0, F, F, 0, F, F, F, F, 0, F, m, 0) == GDR_ERR_NULL_ARG); /* dlog_g of none */
#define BAD(field, value, status)                     \
  t = s;                                              \
  t.field = value;                                    \
  EXPECT(gdr_lin_checkpoint_bytes(&t, &n) == status); \
  EXPECT(lin_fwd(&t, F, F, 0, F, 1) == status);       \
  EXPECT(lin_bwd(&t, F, F, F, F, F, 1) == status)
  BAD(B, -1, GDR_ERR_BAD_DIM);
  BAD(B, 65536, GDR_ERR_BAD_DIM);
  BAD(T, -1, GDR_ERR_BAD_DIM);
  BAD(T, INT64_C(1) << 30, GDR_ERR_BAD_DIM);
  BAD(rows, INT64_C(1) << 30, GDR_ERR_BAD_DIM);
  BAD(Hk, 0, GDR_ERR_BAD_DIM);
  BAD(Hv, 0, GDR_ERR_BAD_DIM);
  BAD(Dk, 0, GDR_ERR_BAD_DIM);
  BAD(Dv, 0, GDR_ERR_BAD_DIM);
  BAD(Hv, 5, GDR_ERR_HEAD_RATIO);
  BAD(Hv, 65536, GDR_ERR_UNSUPPORTED_DIM);
  BAD(Dk, 257, GDR_ERR_UNSUPPORTED_DIM);
  BAD(Dv, 257, GDR_ERR_UNSUPPORTED_DIM);
  BAD(dtype, 2, GDR_ERR_BAD_DTYPE);
  BAD(gdtype, -1, GDR_ERR_BAD_DTYPE);
  BAD(per_head, 2, GDR_ERR_BAD_DECAY);
  BAD(q_stride, 127, GDR_ERR_BAD_STRIDE);
  BAD(k_stride, (INT64_C(1) << 23) + 1, GDR_ERR_BAD_STRIDE);
  BAD(v_stride, 255, GDR_ERR_BAD_STRIDE);
  BAD(g_stride, 3, GDR_ERR_BAD_STRIDE);
#undef BAD
  t = lin(1, 16, 1, 65535, 256, 1, GDR_F32); /* dq of all value heads: rows of 2^24 */
  EXPECT(gdr_lin_checkpoint_bytes(&t, &n) == GDR_ERR_BAD_STRIDE);
  t = s;
  t.rows = 399; /* dense batches own B T rows */
  EXPECT(lin_fwd(&t, F, F, 0, F, 1 << 20) == GDR_ERR_BAD_DIM);
  EXPECT(lin_bwd(&t, F, F, F, F, F, 1 << 30) == GDR_ERR_BAD_DIM);
  t = s;
  t.B = 0; t.rows = 0;
  EXPECT(lin_fwd(&t, 0, 0, 0, 0, 0) == GDR_OK); /* nothing to do */
  EXPECT(lin_bwd(&t, 0, 0, 0, 0, 0, 0) == GDR_OK);
  t = s;
  t.T = 0; t.rows = 0;
  EXPECT(lin_fwd(&t, 0, 0, 0, 0, 0) == GDR_OK); /* no state wanted either */

  gdr_res_shape r = res(64, 96, 16, GDR_BF16), u;
  EXPECT(gdr_res_backward_workspace_bytes(0, &n) == GDR_ERR_NULL_ARG);
  EXPECT(gdr_res_backward_workspace_bytes(&r, 0) == GDR_ERR_NULL_ARG);
  EXPECT(gdr_res_backward_workspace_bytes(&r, &m) == GDR_OK && m > 0);
  EXPECT(res_fwd(&r, 0, F, F) == GDR_ERR_NULL_ARG);
  EXPECT(res_fwd(&r, F, 0, F) == GDR_ERR_NULL_ARG);
  EXPECT(res_fwd(&r, F, F, 0) == GDR_ERR_NULL_ARG);
  EXPECT(res_fwd(&r, M, F, F) == GDR_ERR_ALIGNMENT);
  EXPECT(res_fwd(&r, F, M, F) == GDR_ERR_ALIGNMENT);
  EXPECT(res_bwd(&r, F, 0, F, F, F, F, m) == GDR_ERR_NULL_ARG); /* dy, with the norm of h */
  EXPECT(res_bwd(&r, F, F, M, F, F, F, m) == GDR_ERR_ALIGNMENT);
  EXPECT(res_bwd(&r, F, F, F, F, F, F, m - 1) == GDR_ERR_WORKSPACE);
  EXPECT(res_bwd(&r, F, F, F, F, F, 0, m) == GDR_ERR_WORKSPACE);
  EXPECT(gdr_res_backward(&r, F, F, 0, F, 0, 0, 0, F, F, F, F, F, F, 0, 0, 0, 0, F, m, 0) == GDR_ERR_NULL_ARG); /* dgate of none */
  u = r;
  u.pre = 0;
  EXPECT(res_bwd(&u, F, F, 0, F, F, F, m) == GDR_ERR_NULL_ARG); /* dh, without it */
  u = r;
  u.rows = 0;
  EXPECT(res_fwd(&u, 0, 0, 0) == GDR_OK);
#define BAD(field, value, status)                             \
  u = r;                                                      \
  u.field = value;                                            \
  EXPECT(gdr_res_backward_workspace_bytes(&u, &n) == status); \
  EXPECT(res_fwd(&u, F, F, F) == status);                     \
  EXPECT(res_bwd(&u, F, F, F, F, F, F, 1) == status)
  BAD(rows, -1, GDR_ERR_BAD_DIM);
  BAD(rows, INT64_C(1) << 30, GDR_ERR_BAD_DIM);
  BAD(C, 0, GDR_ERR_BAD_DIM);
  BAD(C, 8193, GDR_ERR_BAD_DIM);
  BAD(gate_rows, -1, GDR_ERR_BAD_DIM);
  BAD(gate_rows, 15, GDR_ERR_BAD_DIM);
  BAD(dtype, 3, GDR_ERR_BAD_DTYPE);
  BAD(rdtype, 3, GDR_ERR_BAD_DTYPE);
  BAD(wdtype, -2, GDR_ERR_BAD_DTYPE);
  BAD(gdtype, 9, GDR_ERR_BAD_DTYPE);
  BAD(post, 2, GDR_ERR_BAD_ACT);
  BAD(pre, -1, GDR_ERR_BAD_ACT);
  BAD(center, 7, GDR_ERR_BAD_ACT);
  BAD(eps, -1e-6f, GDR_ERR_BAD_EPS);
  BAD(eps, INFINITY, GDR_ERR_BAD_EPS);
  BAD(eps, NAN, GDR_ERR_BAD_EPS);
  BAD(x_stride, 95, GDR_ERR_BAD_STRIDE);
  BAD(r_stride, 95, GDR_ERR_BAD_STRIDE);
  BAD(gate_stride, 95, GDR_ERR_BAD_STRIDE);
#undef BAD
  u = res(64, 96, 0, GDR_F32);
  u.rdtype = GDR_BF16; /* a stream narrower than the rows */
  EXPECT(res_fwd(&u, F, F, F) == GDR_ERR_BAD_DTYPE);

  if (fails == 0) printf("block host checks passed\n");
  return fails != 0;
}
