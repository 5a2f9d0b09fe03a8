// Prints, for each shape "B,T,Hk,Hv,Dk,Dv,dtype" given, how the plans of the gated delta rule lay its
// scans out: groups of 16 state columns of a block and segments of a sequence, forward and backward.
#include <stdio.h>

#include "kan_delta.h"

extern "C" hipError_t hipGetLastError(void) { return hipSuccess; }

namespace kan {

hipError_t launch_fill_zero(float*, int64_t, hipStream_t) { return hipSuccess; }
hipError_t launch_delta_fwd(const kan_delta_desc_t&, const DeltaPlan&, const DeltaArgs&, char*, hipStream_t) {
    return hipSuccess;
}
hipError_t launch_delta_bwd(const kan_delta_desc_t&, const DeltaPlan&, const DeltaArgs&, char*, hipStream_t) {
    return hipSuccess;
}
hipError_t launch_delta_step(const kan_delta_desc_t&, int64_t, const DeltaArgs&, float*, const int32_t*, hipStream_t) {
    return hipSuccess;
}
hipError_t launch_join_fwd(const kan_join_desc_t&, const JoinPlan&, const JoinArgs&, hipStream_t) { return hipSuccess; }
hipError_t launch_join_bwd(const kan_join_desc_t&, const JoinPlan&, const JoinArgs&, char*, hipStream_t) {
    return hipSuccess;
}

}  // namespace kan

int main(int argc, char** argv) {
    for (int i = 1; i < argc; ++i) {
        kan_delta_desc_t d = {};
        if (sscanf(argv[i], "%ld,%ld,%ld,%ld,%ld,%ld,%d", &d.B, &d.T, &d.Hk, &d.Hv, &d.Dk, &d.Dv, &d.dtype) != 7) return 1;
        const kan::DeltaPlan f = kan::delta_plan(d, KAN_PASS_FORWARD), b = kan::delta_plan(d, KAN_PASS_BACKWARD);
        printf("%d %d %d %d %d\n", f.dkp, f.groups, f.segs, b.groups, b.segs);
    }
    return 0;
}
