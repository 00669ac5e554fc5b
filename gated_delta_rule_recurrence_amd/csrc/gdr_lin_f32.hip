// The chunked linear attention's instances for f32 rows
// (see gdr_lin.h).
#include "gdr_lin_launch.h"

namespace gdr {
template hipError_t lin_chunk<float, true>(const LinArgs& a, const LinRole& r, int mode,
                                    hipStream_t s);
template hipError_t lin_chunks<float, true>(const LinArgs& a, const LinRoles& r, int mode,
                                     hipStream_t s);
}  // namespace gdr
