// Products in 8-bit floating point whose scales are powers of two and whose outputs are float32.
#include "gq_mm_tile.h"

namespace gq {

hipError_t mm_launch_e8w(MmForm form, const MmTile& t, const MmPlan& P, hipStream_t st) {
    if (form == MM_NT) return mm_launch_rows<MM_E8W, MM_NT>(t, P, st);
    if (form == MM_GATE) return mm_launch_rows<MM_E8W, MM_GATE>(t, P, st);
    return mm_launch_back<MM_E8W>(t, P, st);
}

}  // namespace gq
