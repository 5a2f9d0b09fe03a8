// Status of kan_delta_backward for gradients that share one array, with launchers that do nothing.
// Arguments: B,T,Hk,Hv,Dk,Dv, then for each of dq, dk, dv its place in the array and its strides of
// sequences, rows and heads (elements of float32).
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

template <typename T = void>
static T* at(int k) {
    return reinterpret_cast<T*>((uintptr_t)(k + 1) << 40);
}

int main(int argc, char** argv) {
    for (int i = 1; i < argc; ++i) {
        kan_delta_desc_t d = {};
        long o[3];
        kan_heads_t s[3];
        if (sscanf(argv[i], "%ld,%ld,%ld,%ld,%ld,%ld,%ld,%ld,%ld,%ld,%ld,%ld,%ld,%ld,%ld,%ld,%ld,%ld", &d.B, &d.T, &d.Hk,
                   &d.Hv, &d.Dk, &d.Dv, &o[0], &s[0].seq, &s[0].row, &s[0].head, &o[1], &s[1].seq, &s[1].row, &s[1].head,
                   &o[2], &s[2].seq, &s[2].row, &s[2].head) != 18)
            return 1;
        d.q = d.k = kan_heads_t{d.T * d.Hk * d.Dk, d.Hk * d.Dk, d.Dk};
        d.v = kan_heads_t{d.T * d.Hv * d.Dv, d.Hv * d.Dv, d.Dv};
        d.dq = s[0], d.dk = s[1], d.dv = s[2];
        d.scale = 1.0f;
        float* const p = at<float>(15);
        printf("%d\n", kan_delta_backward(&d, at(0), at(1), at(2), at<float>(3), at<float>(4), at<float>(5),
                                          at<int32_t>(6), at(7), at<float>(8), p + o[0], p + o[1], p + o[2], at<float>(9),
                                          at<float>(10), at<float>(11), at(12), size_t(1) << 39, nullptr));
    }
    return 0;
}
