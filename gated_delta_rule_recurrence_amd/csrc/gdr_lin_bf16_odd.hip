// The chunked linear attention's instances for bf16 rows that are not whole vectors
// (see gdr_lin.h).
#include "gdr_lin_launch.h"

namespace gdr {
template hipError_t lin_chunk<bf16, false>(const LinArgs& a, const LinRole& r, int mode,
                                    hipStream_t s);
template hipError_t lin_chunks<bf16, false>(const LinArgs& a, const LinRoles& r, int mode,
                                     hipStream_t s);
}  // namespace gdr
