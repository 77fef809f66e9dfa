// The gated feed-forward block's products with bfloat16 weights.
#include "gq_mm_tile.h"

namespace gq {

hipError_t mm_launch_bf16(MmForm form, const MmTile& t, const MmPlan& P, hipStream_t st) {
    if (form == MM_GATE) return mm_launch_rows<MM_BF16, MM_GATE>(t, P, st);
    if (form == MM_NN) return mm_launch_back<MM_BF16>(t, P, st);
    return P.bm == 256 ? mm_launch_tile<MM_BF16, MM_TN, 256, 256, 4, 8, 2>(t, P, st)
                       : mm_launch_tile<MM_BF16, MM_TN, 128, 128, 2, 4, 2>(t, P, st);
}

}  // namespace gq
