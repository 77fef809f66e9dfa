// Products in 8-bit floating point whose scales are powers of two, which the matrix cores apply.
#include "gq_mm_tile.h"

namespace gq {

hipError_t mm_launch_e8(MmForm form, const MmTile& t, const MmPlan& P, hipStream_t st) {
    if (form == MM_NT) return mm_launch_rows<MM_E8, MM_NT>(t, P, st);
    if (form == MM_GATE) return mm_launch_rows<MM_E8, MM_GATE>(t, P, st);
    return mm_launch_back<MM_E8>(t, P, st);
}

}  // namespace gq
