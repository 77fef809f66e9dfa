// Products in 8-bit floating point whose scales are float32 numbers and whose outputs are float32.
#include "gq_mm_tile.h"

namespace gq {

hipError_t mm_launch_fsw(MmForm form, const MmTile& t, const MmPlan& P, hipStream_t st) {
    if (form == MM_NT) return mm_launch_rows<MM_FSW, MM_NT>(t, P, st);
    if (form == MM_GATE) return mm_launch_rows<MM_FSW, MM_GATE>(t, P, st);
    return mm_launch_back<MM_FSW>(t, P, st);
}

}  // namespace gq
