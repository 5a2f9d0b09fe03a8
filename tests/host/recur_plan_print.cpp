// Host program: the launch plans of the gated recurrence (recur_plan in
// kan_token_api.cpp).  For each group of arguments B T D dtype grad_dtype packed
// one line for each pass: channels of a lane, lanes, waves, segments, rows of a
// segment, rows of a tile, whether rows start on cache lines.
#include <stdio.h>
#include <stdlib.h>

#include "kan_token.h"

extern "C" hipError_t hipGetLastError(void) { return hipSuccess; }

namespace kan {

// kan_token_api.cpp's launchers; nothing is launched here
hipError_t launch_fill_zero(float*, int64_t, hipStream_t) { return hipErrorUnknown; }
hipError_t launch_embed_fwd(const kan_embed_desc_t&, const void*, const void*, void*, hipStream_t) {
    return hipErrorUnknown;
}
hipError_t launch_embed_bwd(const kan_embed_desc_t&, const EmbedPlan&, const void*, const void*, float*, char*,
                            hipStream_t) {
    return hipErrorUnknown;
}
hipError_t launch_recur_fwd(const kan_recur_desc_t&, const RecurPlan&, const RecurArgs&, char*, hipStream_t) {
    return hipErrorUnknown;
}
hipError_t launch_recur_bwd(const kan_recur_desc_t&, const RecurPlan&, const RecurArgs&, char*, hipStream_t) {
    return hipErrorUnknown;
}
hipError_t launch_recur_step(const kan_recur_desc_t&, int64_t, const void*, const void*, float*, const int32_t*, float*,
                             hipStream_t) {
    return hipErrorUnknown;
}
hipError_t launch_distill(const kan_distill_desc_t&, const DistillPlan&, const DistillArgs&, char*, hipStream_t) {
    return hipErrorUnknown;
}
hipError_t launch_distill_bwd(const kan_distill_desc_t&, const DistillArgs&, hipStream_t) { return hipErrorUnknown; }

}  // namespace kan

int main(int argc, char** argv) {
    for (int i = 1; i + 5 < argc; i += 6) {
        const int64_t B = atoll(argv[i]), T = atoll(argv[i + 1]), D = atoll(argv[i + 2]);
        const int64_t row = atoi(argv[i + 5]) ? 2 * D : D;
        const kan_recur_desc_t d{B,   T,       D,   row,     row * T, row,
                                 row * T, row, row * T, row, row * T, atoi(argv[i + 3]), atoi(argv[i + 4])};
        for (int pass : {KAN_PASS_FORWARD, KAN_PASS_BACKWARD}) {
            const kan::RecurPlan p = kan::recur_plan(d, pass);
            printf("%d %d %d %d %lld %d %d\n", p.vec, p.lanes, p.waves, p.segs, (long long)p.seg_rows,
                   p.waves * kan::kRecurRows * (64 / p.lanes), (int)p.on_lines);
        }
    }
    return 0;
}
