// The chunked linear attention's instances for f32 rows that are not whole vectors
// (see gdr_lin.h).
#include "gdr_lin_launch.h"

namespace gdr {
template hipError_t lin_chunk<float, false>(const LinArgs& a, const LinRole& r, int mode,
                                    hipStream_t s);
template hipError_t lin_chunks<float, false>(const LinArgs& a, const LinRoles& r, int mode,
                                     hipStream_t s);
}  // namespace gdr
