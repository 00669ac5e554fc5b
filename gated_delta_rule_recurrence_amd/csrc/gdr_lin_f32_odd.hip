// The chunked linear attention's instances for f32 rows that are not whole vectors
// (see gdr_lin.h).
#include "gdr_lin_launch.h"

namespace gdr {
template hipError_t lin_chunk<float, false>(const LinArgs& a, LinRole r, int mode, hipStream_t s);
}  // namespace gdr
