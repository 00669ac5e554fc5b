// Choice of the chunked linear attention's instance (see gdr_lin.h).
#pragma once

#include "gdr_lin.h"

namespace gdr {

template <typename T, int KI, int NT, int MODE, bool VEC>
hipError_t lin_launch(const LinArgs& a, const LinRole& r, hipStream_t s) {
  hipLaunchKernelGGL((lin_chunk_kernel<T, KI, NT, MODE, VEC>),
                     dim3((unsigned)r.tiles * a.segs, a.Hv, a.B), dim3(256), 0, s, a, r);
  const hipError_t e = hipGetLastError();
  note_launch(s);
  return e;
}
template <typename T, int KI, int NT, bool VEC>
hipError_t lin_mode(const LinArgs& a, const LinRole& r, int mode, hipStream_t s) {
  if (mode == kLinOut) return lin_launch<T, KI, NT, kLinOut, VEC>(a, r, s);
  if (mode == kLinFlow) return lin_launch<T, KI, NT, kLinFlow, VEC>(a, r, s);
  return lin_launch<T, KI, NT, kLinState, VEC>(a, r, s);
}
template <typename T, int KI, bool VEC>
hipError_t lin_wide(const LinArgs& a, const LinRole& r, int mode, hipStream_t s) {
  if constexpr (KI <= 128)
    if (lin_width(r.Ni, r.No) == 128) return lin_mode<T, KI, 2, VEC>(a, r, mode, s);
  return lin_mode<T, KI, 1, VEC>(a, r, mode, s);
}
template <typename T, bool VEC>
hipError_t lin_chunk(const LinArgs& a, const LinRole& r, int mode, hipStream_t s) {
  if (r.Ni <= 64) return lin_wide<T, 64, VEC>(a, r, mode, s);
  if (r.Ni <= 128) return lin_wide<T, 128, VEC>(a, r, mode, s);
  if (r.Ni <= 192) return lin_wide<T, 192, VEC>(a, r, mode, s);
  return lin_wide<T, 256, VEC>(a, r, mode, s);
}

template <typename T, int KI, int NT, int MODE, bool VEC>
hipError_t lin_launch3(const LinArgs& a, const LinRoles& r, hipStream_t s) {
  hipLaunchKernelGGL((lin_chunks_kernel<T, KI, NT, MODE, VEC>),
                     dim3((unsigned)r.r[0].tiles * a.segs * 3, a.Hv, a.B), dim3(256), 0, s, a,
                     r);
  const hipError_t e = hipGetLastError();
  note_launch(s);
  return e;
}
template <typename T, int KI, int NT, bool VEC>
hipError_t lin_mode3(const LinArgs& a, const LinRoles& r, int mode, hipStream_t s) {
  return mode == kLinOut ? lin_launch3<T, KI, NT, kLinOut, VEC>(a, r, s)
                         : lin_launch3<T, KI, NT, kLinFlow, VEC>(a, r, s);
}
// One launch for widths of up to 64, or of 65 to 128, on both sides; else one
// each.
template <typename T, bool VEC>
hipError_t lin_chunks(const LinArgs& a, const LinRoles& r, int mode, hipStream_t s) {
  const int n = a.Dk < a.Dv ? a.Dk : a.Dv, m = a.Dk < a.Dv ? a.Dv : a.Dk;
  if (m <= 64) return lin_mode3<T, 64, 1, VEC>(a, r, mode, s);
  if (n > 64 && m <= 128) return lin_mode3<T, 128, 2, VEC>(a, r, mode, s);
  hipError_t e = lin_chunk<T, VEC>(a, r.r[0], mode, s);
  if (e == hipSuccess) e = lin_chunk<T, VEC>(a, r.r[1], mode, s);
  return e == hipSuccess ? lin_chunk<T, VEC>(a, r.r[2], kLinOut, s) : e;
}

}  // namespace gdr
