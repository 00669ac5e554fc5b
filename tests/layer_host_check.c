/* Host-side checks of the convolution's, the scan's and the norm's C entry
 * points (include/gdr.h) for a sanitizer build: the size queries over many
 * shapes, up to the limits, and every argument-rejection path.  Nothing here
 * reaches the device: every call either only computes sizes or is rejected
 * on the host.  Exits non-zero on the first wrong status.  Built and run by
 * tests/test_layer_abi.py. */
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

static gdr_conv_shape conv(int64_t B, int64_t T, int64_t C, int64_t K, int32_t dt) {
  gdr_conv_shape s;
  memset(&s, 0, sizeof s);
  s.B = B; s.T = T; s.rows = B * T; s.C = C; s.K = K; s.dtype = dt; s.wdtype = dt;
  s.act = GDR_ACT_SILU;
  return s;
}
static gdr_scan_shape scan(int64_t B, int64_t T, int64_t C, int64_t N, int64_t G, int32_t dt) {
  gdr_scan_shape s;
  memset(&s, 0, sizeof s);
  s.B = B; s.T = T; s.rows = B * T; s.C = C; s.N = N; s.G = G; s.dtype = dt; s.softplus = 1;
  return s;
}
static gdr_norm_shape norm(int64_t rows, int64_t C, int64_t G, int32_t dt) {
  gdr_norm_shape s;
  memset(&s, 0, sizeof s);
  s.rows = rows; s.C = C; s.G = G; s.dtype = dt; s.wdtype = dt; s.eps = 1e-6f;
  return s;
}

int main(void) {
  static char buf[64] __attribute__((aligned(16)));
  void* F = buf;
  void* M = buf + 4; /* misaligned */
  size_t n = 0;
  const int64_t Ts[] = {0, 1, 15, 16, 17, 300, 8192, (INT64_C(1) << 30) - 1};
  const int64_t Cs[] = {1, 7, 64, 65, 4096, 8192, INT64_C(1) << 20};
  for (size_t i = 0; i < sizeof Ts / sizeof Ts[0]; ++i)
    for (size_t j = 0; j < sizeof Cs / sizeof Cs[0]; ++j)
      for (int dt = 0; dt < 2; ++dt) {
        gdr_conv_shape c = conv(1, Ts[i], Cs[j], 8, dt);
        int st = gdr_conv_backward_workspace_bytes(&c, &n);
        EXPECT(st == GDR_OK || st == GDR_ERR_OVERFLOW);
        for (int64_t N = 1; N <= 64; N *= 4) {
          gdr_scan_shape s = scan(1, Ts[i], Cs[j], N, 1, dt);
          st = gdr_scan_checkpoint_bytes(&s, &n);
          EXPECT(st == GDR_OK || st == GDR_ERR_OVERFLOW);
          st = gdr_scan_forward_workspace_bytes(&s, &n);
          EXPECT(st == GDR_OK || st == GDR_ERR_OVERFLOW);
          st = gdr_scan_backward_workspace_bytes(&s, &n);
          EXPECT(st == GDR_OK || st == GDR_ERR_OVERFLOW);
        }
        for (int64_t G = 1; G <= Cs[j]; G *= 3) {
          if (Cs[j] % G) continue;
          gdr_norm_shape m = norm(Ts[i], Cs[j], G, dt);
          st = gdr_norm_backward_workspace_bytes(&m, &n);
          const int64_t D = Cs[j] / G;
          EXPECT(st == (Ts[i] * G > INT32_MAX ? GDR_ERR_OVERFLOW
                                              : D > 8192 ? GDR_ERR_BAD_DIM : GDR_OK));
        }
      }

  /* convolution: shapes, pointers, alignment, workspace */
  gdr_conv_shape c = conv(2, 8, 16, 4, GDR_F32);
#define CF(s, x, w, b, st, sp, y, so) gdr_conv_forward(s, x, w, b, st, sp, y, so, NULL)
  EXPECT(CF(NULL, F, F, F, F, NULL, F, F) == GDR_ERR_NULL_ARG);
  c.K = 0; EXPECT(CF(&c, F, F, F, F, NULL, F, F) == GDR_ERR_BAD_DIM);
  c.K = 9; EXPECT(CF(&c, F, F, F, F, NULL, F, F) == GDR_ERR_BAD_DIM);
  c = conv(2, 8, 16, 4, GDR_F32); c.C = 0; EXPECT(CF(&c, F, F, F, F, NULL, F, F) == GDR_ERR_BAD_DIM);
  c.C = (1 << 20) + 1; EXPECT(CF(&c, F, F, F, F, NULL, F, F) == GDR_ERR_BAD_DIM);
  c = conv(2, 8, 16, 4, GDR_F32); c.B = 65536; EXPECT(CF(&c, F, F, F, F, F, F, F) == GDR_ERR_BAD_DIM);
  c = conv(2, 8, 16, 4, GDR_F32); c.T = -1; EXPECT(CF(&c, F, F, F, F, F, F, F) == GDR_ERR_BAD_DIM);
  c = conv(2, 8, 16, 4, GDR_F32); c.rows = 15; EXPECT(CF(&c, F, F, F, F, NULL, F, F) == GDR_ERR_BAD_DIM);
  c = conv(2, 8, 16, 4, GDR_F32); c.dtype = 2; EXPECT(CF(&c, F, F, F, F, NULL, F, F) == GDR_ERR_BAD_DTYPE);
  c = conv(2, 8, 16, 4, GDR_F32); c.wdtype = -1; EXPECT(CF(&c, F, F, F, F, NULL, F, F) == GDR_ERR_BAD_DTYPE);
  c = conv(2, 8, 16, 4, GDR_F32); c.act = 2; EXPECT(CF(&c, F, F, F, F, NULL, F, F) == GDR_ERR_BAD_ACT);
  c = conv(2, 8, 16, 4, GDR_F32); c.x_stride = 15; EXPECT(CF(&c, F, F, F, F, NULL, F, F) == GDR_ERR_BAD_STRIDE);
  c.x_stride = INT64_C(1) << 31; EXPECT(CF(&c, F, F, F, F, NULL, F, F) == GDR_ERR_BAD_STRIDE);
  c = conv(2, 8, 16, 4, GDR_F32);
  EXPECT(CF(&c, NULL, F, F, F, NULL, F, F) == GDR_ERR_NULL_ARG);
  EXPECT(CF(&c, F, NULL, F, F, NULL, F, F) == GDR_ERR_NULL_ARG);
  EXPECT(CF(&c, F, F, F, F, NULL, NULL, F) == GDR_ERR_NULL_ARG);
  EXPECT(CF(&c, M, F, F, F, NULL, F, F) == GDR_ERR_ALIGNMENT);
  EXPECT(CF(&c, F, F, F, F, M, F, F) == GDR_ERR_ALIGNMENT);
  EXPECT(CF(&c, F, F, F, F, NULL, F, M) == GDR_ERR_ALIGNMENT);
  c = conv(0, 8, 16, 4, GDR_F32); EXPECT(CF(&c, NULL, NULL, NULL, NULL, NULL, NULL, NULL) == GDR_OK);
  c = conv(2, 0, 16, 4, GDR_F32); EXPECT(CF(&c, NULL, NULL, NULL, NULL, NULL, NULL, NULL) == GDR_OK);
  EXPECT(CF(&c, NULL, NULL, NULL, NULL, NULL, NULL, F) == GDR_ERR_NULL_ARG);
  c = conv(2, 8, 16, 4, GDR_F32);
  EXPECT(gdr_conv_backward_workspace_bytes(&c, NULL) == GDR_ERR_NULL_ARG);
  EXPECT(gdr_conv_backward_workspace_bytes(&c, &n) == GDR_OK && n > 0);
#define CB(ws, by, dx, dw) gdr_conv_backward(&c, F, F, F, F, NULL, F, F, dx, dw, F, F, ws, by, NULL)
  EXPECT(CB(F, n - 1, F, F) == GDR_ERR_WORKSPACE);
  EXPECT(CB(NULL, n, F, F) == GDR_ERR_NULL_ARG);
  EXPECT(CB(F, n, NULL, F) == GDR_ERR_NULL_ARG);
  EXPECT(CB(F, n, F, NULL) == GDR_ERR_NULL_ARG);
  EXPECT(CB(M, n, F, F) == GDR_ERR_ALIGNMENT);
  c = conv(0, 8, 16, 4, GDR_F32);
  EXPECT(gdr_conv_backward(&c, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL,
                           NULL, 0, NULL) == GDR_OK);

  /* scan */
  gdr_scan_shape s = scan(1, 300, 64, 16, 2, GDR_BF16);
  float* P = (float*)F;
#define SF(sh, u, A, y, ws, by) \
  gdr_scan_forward(sh, u, F, A, F, F, P, F, P, P, NULL, y, P, F, ws, by, NULL)
  EXPECT(SF(NULL, F, P, F, F, 1 << 30) == GDR_ERR_NULL_ARG);
  s.N = 65; EXPECT(SF(&s, F, P, F, F, 1 << 30) == GDR_ERR_BAD_DIM);
  s.N = 0; EXPECT(SF(&s, F, P, F, F, 1 << 30) == GDR_ERR_BAD_DIM);
  s = scan(1, 300, 64, 16, 3, GDR_BF16); EXPECT(SF(&s, F, P, F, F, 1 << 30) == GDR_ERR_BAD_DIM);
  s = scan(1, 300, 64, 16, 0, GDR_BF16); EXPECT(SF(&s, F, P, F, F, 1 << 30) == GDR_ERR_BAD_DIM);
  s = scan(1, 300, 64, 16, 2, 7); EXPECT(SF(&s, F, P, F, F, 1 << 30) == GDR_ERR_BAD_DTYPE);
  s = scan(1, 300, 64, 16, 2, GDR_BF16); s.softplus = 2;
  EXPECT(SF(&s, F, P, F, F, 1 << 30) == GDR_ERR_BAD_ACT);
  s = scan(1, 300, 64, 16, 2, GDR_BF16); s.b_stride = 31;
  EXPECT(SF(&s, F, P, F, F, 1 << 30) == GDR_ERR_BAD_STRIDE);
  s = scan(1, 300, 64, 16, 2, GDR_BF16); s.rows = 301;
  EXPECT(SF(&s, F, P, F, F, 1 << 30) == GDR_ERR_BAD_DIM);
  s = scan(1, 300, 64, 16, 2, GDR_BF16);
  EXPECT(SF(&s, NULL, P, F, F, 1 << 30) == GDR_ERR_NULL_ARG);
  EXPECT(SF(&s, F, NULL, F, F, 1 << 30) == GDR_ERR_NULL_ARG);
  EXPECT(SF(&s, F, P, NULL, F, 1 << 30) == GDR_ERR_NULL_ARG);
  EXPECT(SF(&s, F, P, M, F, 1 << 30) == GDR_ERR_ALIGNMENT);
  EXPECT(gdr_scan_forward_workspace_bytes(&s, &n) == GDR_OK && n > 0);
  EXPECT(SF(&s, F, P, F, F, n - 1) == GDR_ERR_WORKSPACE);
  EXPECT(SF(&s, F, P, F, NULL, n) == GDR_ERR_WORKSPACE);
  EXPECT(gdr_scan_checkpoint_bytes(&s, NULL) == GDR_ERR_NULL_ARG);
  EXPECT(gdr_scan_backward_workspace_bytes(&s, &n) == GDR_OK && n > 0);
#define SB(dA, dz, ck, ws, by) \
  gdr_scan_backward(&s, F, F, P, F, F, P, F, P, NULL, ck, F, P, F, F, dA, F, F, P, dz, P, P, ws, by, NULL)
  EXPECT(SB(P, F, F, F, n - 1) == GDR_ERR_WORKSPACE);
  EXPECT(SB(NULL, F, F, F, n) == GDR_ERR_NULL_ARG);
  EXPECT(SB(P, NULL, F, F, n) == GDR_ERR_NULL_ARG);
  EXPECT(SB(P, F, NULL, F, n) == GDR_ERR_NULL_ARG);
  EXPECT(SB(P, F, F, NULL, n) == GDR_ERR_NULL_ARG);
  EXPECT(SB(P, M, F, F, n) == GDR_ERR_ALIGNMENT);
  s = scan(0, 300, 64, 16, 2, GDR_BF16);
  EXPECT(SF(&s, NULL, NULL, NULL, NULL, 0) == GDR_OK);
  s = scan(65535, (INT64_C(1) << 30) - 1, 1 << 20, 64, 1, GDR_BF16);
  s.rows = (INT64_C(1) << 30) - 1;
  EXPECT(gdr_scan_backward_workspace_bytes(&s, &n) == GDR_ERR_OVERFLOW);

  /* norm */
  gdr_norm_shape m = norm(4, 60, 3, GDR_F32);
#define NF(sh, x, w, y, st) gdr_norm_forward(sh, x, w, F, F, y, st, NULL)
  EXPECT(NF(NULL, F, F, F, P) == GDR_ERR_NULL_ARG);
  m.G = 7; EXPECT(NF(&m, F, F, F, P) == GDR_ERR_BAD_DIM);
  m = norm(4, 60, 0, GDR_F32); EXPECT(NF(&m, F, F, F, P) == GDR_ERR_BAD_DIM);
  m = norm(4, 8193, 1, GDR_F32); EXPECT(NF(&m, F, F, F, P) == GDR_ERR_BAD_DIM);
  m = norm(-1, 60, 3, GDR_F32); EXPECT(NF(&m, F, F, F, P) == GDR_ERR_BAD_DIM);
  m = norm(4, 60, 3, 5); EXPECT(NF(&m, F, F, F, P) == GDR_ERR_BAD_DTYPE);
  m = norm(4, 60, 3, GDR_F32); m.act = -1; EXPECT(NF(&m, F, F, F, P) == GDR_ERR_BAD_ACT);
  m = norm(4, 60, 3, GDR_F32); m.eps = -1.f; EXPECT(NF(&m, F, F, F, P) == GDR_ERR_BAD_EPS);
  m.eps = NAN; EXPECT(NF(&m, F, F, F, P) == GDR_ERR_BAD_EPS);
  m.eps = INFINITY; EXPECT(NF(&m, F, F, F, P) == GDR_ERR_BAD_EPS);
  m = norm(4, 60, 3, GDR_F32); m.z_stride = 59; EXPECT(NF(&m, F, F, F, P) == GDR_ERR_BAD_STRIDE);
  m = norm(4, 60, 3, GDR_F32);
  EXPECT(NF(&m, NULL, F, F, P) == GDR_ERR_NULL_ARG);
  EXPECT(NF(&m, F, F, NULL, P) == GDR_ERR_NULL_ARG);
  EXPECT(NF(&m, F, M, F, P) == GDR_ERR_ALIGNMENT);
  EXPECT(gdr_norm_backward_workspace_bytes(&m, &n) == GDR_OK && n > 0);
#define NB(st, dx, dz, ws, by) gdr_norm_backward(&m, F, F, F, F, st, F, dx, F, F, dz, ws, by, NULL)
  EXPECT(NB(P, F, F, F, n - 1) == GDR_ERR_WORKSPACE);
  EXPECT(NB(P, F, F, NULL, n) == GDR_ERR_WORKSPACE);
  EXPECT(NB(NULL, F, F, F, n) == GDR_ERR_NULL_ARG);
  EXPECT(NB(P, NULL, F, F, n) == GDR_ERR_NULL_ARG);
  EXPECT(NB(P, F, NULL, F, n) == GDR_ERR_NULL_ARG);
  EXPECT(NB(P, F, M, F, n) == GDR_ERR_ALIGNMENT);
  m = norm(0, 60, 3, GDR_F32); EXPECT(NF(&m, NULL, NULL, NULL, NULL) == GDR_OK);

  for (int code = 0; code >= GDR_ERR_BAD_EPS; --code)
    EXPECT(strstr(gdr_strerror(code), "unknown") == NULL);
  if (fails) return 1;
  printf("layer host checks passed\n");
  return 0;
}
