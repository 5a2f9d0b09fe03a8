// Host-only run of the validation and planning of the gated delta rule and the
// join (kan_delta_api.cpp) under AddressSanitizer and UndefinedBehaviorSanitizer.
// Launcher stubs check what every launcher relies on: plans that cover the work,
// carve-outs that lie one behind the other inside the declared workspace, grids
// inside the limits of a launch.  Exit status 0 and "ok": everything held.
#include <stdio.h>
#include <stdlib.h>

#include <initializer_list>

#include "kan_delta.h"

static long launches = 0;
static size_t ws_bytes = 0;

extern "C" hipError_t hipGetLastError(void) { return hipSuccess; }

static void need(bool ok, const char* what) {
    if (!ok) {
        fprintf(stderr, "check failed: %s\n", what);
        abort();
    }
}

namespace kan {

constexpr int64_t kGrid = (int64_t(1) << 32) - 1;     // threads of a launch

hipError_t launch_fill_zero(float* p, int64_t n, hipStream_t) {
    need(p && n >= 0, "fill");
    ++launches;
    return hipSuccess;
}
static void delta(const kan_delta_desc_t& d, const DeltaPlan& p, const char* ws, bool back) {
    need(p.dkp >= d.Dk && (p.dkp == 32 || p.dkp == 64 || p.dkp == 128) && p.dvp >= d.Dv && p.dvp % 64 == 0, "widths");
    need(p.chunks * kDeltaChunk >= d.T && (p.chunks - 1) * kDeltaChunk < d.T && p.heads == d.B * d.Hv, "chunks");
    need(p.groups == 2 || p.groups == 4, "groups");
    need(p.segs >= 1 && (int64_t)p.segs * p.seg_chunks >= p.chunks, "segments cover the chunks");
    need(p.segs == 1 || ((int64_t)(p.segs - 1) * p.seg_chunks < p.chunks && p.groups == 2), "no empty segment");
    need(p.segs == 1 || p.runs == p.segs - (back ? 0 : 1), "runs");
    // parts of the workspace, in their order
    const int64_t ch = p.heads * p.chunks, sg = p.heads * p.segs;
    size_t at = 0;
    auto part = [&](size_t off, int64_t n, int64_t bytes) {
        need(off >= at && off % 256 == 0, "parts of the workspace");
        at = off + (size_t)(n * bytes);
    };
    part(p.off_rows, ch, 8 * 64 * 4);
    part(p.off_mats, ch, p.mats);
    if (back) {
        part(p.off_w, ch, 64 * p.dvp * 4);
        part(p.off_r, ch, 64 * p.dvp * 4);
        part(p.off_S, ch, (int64_t)p.dkp * p.dvp * 4);
        part(p.off_dS, ch, (int64_t)p.dkp * p.dvp * 4);
        if (d.Hv > d.Hk) {
            part(p.off_dq, d.B * d.T * d.Hv, d.Dk * 4);
            part(p.off_dk, d.B * d.T * d.Hv, d.Dk * 4);
        }
    }
    if (p.segs > 1) {
        part(p.off_runs, sg, (int64_t)p.dkp * (p.dvp + p.dkp) * 4);
        part(p.off_starts, sg, (int64_t)p.dkp * p.dvp * 4);
        if (back) part(p.off_ends, sg, (int64_t)p.dkp * p.dvp * 4);
    }
    need(at <= p.ws && (d.T == 0 || (p.ws <= ws_bytes && ws)), "workspace");
    // grids: threads of the widest blocks of each kernel, counters of blocks in 32 bits
    const int64_t narrow = (d.Dv + 31) / 32, wide = (d.Dv + 63) / 64;
    need(d.B * d.Hk * p.chunks * 256 <= kGrid && ch * 256 <= kGrid, "grids of chunks");
    need(sg * (p.groups == 2 || back ? narrow : wide) * 256 <= kGrid, "grid of a scan");
    if (p.segs > 1)
        need(p.heads * p.runs * (narrow + p.dkp / 32) * 256 <= kGrid && p.heads * ((d.Dv + 15) / 16) * 512 <= kGrid,
             "grids of the runs and their link");
    const int64_t rows = (d.B * d.T * d.Hk + 3) / 4;
    need((rows + 65535) / 65536 <= 65535, "grid of the heads' sums");
    ++launches;
}
hipError_t launch_delta_fwd(const kan_delta_desc_t& d, const DeltaPlan& p, const DeltaArgs& a, char* ws, hipStream_t) {
    need(d.B > 0 && a.q && a.k && a.v && a.g && a.beta && a.y && a.hT, "forward pointers");
    delta(d, p, ws, false);
    return hipSuccess;
}
hipError_t launch_delta_bwd(const kan_delta_desc_t& d, const DeltaPlan& p, const DeltaArgs& a, char* ws, hipStream_t) {
    need(d.B > 0 && a.q && a.k && a.v && a.g && a.beta && a.dy && a.dq && a.dk && a.dv && a.dg && a.dbeta && a.dh0,
         "backward pointers");
    delta(d, p, ws, true);
    return hipSuccess;
}
hipError_t launch_delta_step(const kan_delta_desc_t& d, int64_t S, const DeltaArgs& a, float* state,
                             const int32_t* slots, hipStream_t) {
    need(d.T == 1 && a.q && a.k && a.v && a.g && a.beta && a.y && state && (slots || S >= d.B), "step");
    need(d.B * d.Hv * ((d.Dv + 63) / 64) * 256 <= kGrid, "step grid");
    ++launches;
    return hipSuccess;
}
static void join(const kan_join_desc_t& d, const JoinPlan& p, bool back) {
    need(d.N > 0 && (int64_t)p.lanes * p.vecs * 4 >= d.D, "a row's threads hold it");
    need((p.lanes == 32 && p.vecs == 1) || (p.lanes == 64 && p.vecs <= (back ? 2 : 4)) ||
             (p.lanes == 256 && p.vecs >= (back ? 1 : 2)) || (p.lanes == 1024 && p.vecs == 2),
         "threads of a row");
    need(p.vecs == 1 || p.vecs == 2 || p.vecs == 4, "vectors of a thread");
    need((int64_t)p.blocks * (p.lanes > 256 ? p.lanes : 256) <= kGrid, "join grid");
}
hipError_t launch_join_fwd(const kan_join_desc_t& d, const JoinPlan& p, const JoinArgs& a, hipStream_t) {
    join(d, p, false);
    need(a.h && a.y && a.stats && a.x, "join forward pointers");
    need(p.rows == 1 || (p.rows == kJoinRows && p.vecs == 1), "rows of a thread");
    need((int64_t)p.blocks * p.rows * (p.lanes > 256 ? 1 : 256 / p.lanes) >= d.N, "a pass over the rows");
    ++launches;
    return hipSuccess;
}
hipError_t launch_join_bwd(const kan_join_desc_t& d, const JoinPlan& p, const JoinArgs& a, char* ws, hipStream_t) {
    join(d, p, true);
    need(a.h && a.y_in && a.stats_in && a.dh && ws, "join backward pointers");
    need(p.blocks <= kJoinMaxBlocks && (size_t)p.blocks * 2 * d.D * 4 <= ws_bytes, "blocks' sums fit");
    ++launches;
    return hipSuccess;
}

}  // namespace kan

template <typename T = void>
static T* at(int k) {
    return reinterpret_cast<T*>((uintptr_t)(k + 1) << 52);
}

int main() {
    const size_t big = size_t(1) << 51;
    long want = 0;
    for (int64_t B : {0, 1, 7, 64, 1000, 1 << 18})
        for (int64_t T : {0, 1, 63, 64, 65, 777, 1531, 4096, 32768, 1000003, 1 << 29})
            for (int64_t Hv : {1, 2, 8, 16, 255, 256, 257, 1 << 18})
                for (int64_t Dk : {1, 32, 33, 64, 65, 128})
                    for (int64_t Dv : {1, 32, 33, 64, 104, 128, 1000, 1024})
                        for (int32_t dtype : {KAN_F32, KAN_BF16}) {
                            const int64_t Hk = Hv % 2 ? Hv : Hv / 2, kr = Hk * Dk, vr = Hv * Dv;
                            const kan_heads_t k{T * kr, kr, Dk}, v{T * vr, vr, Dv};
                            kan_delta_desc_t d{B, T, Hk, Hv, Dk, Dv, k, k, v, k, k, v, dtype, KAN_DELTA_UNIT, 0.5f};
                            const int64_t chunks = (T + 63) / 64;
                            const bool fits = B * Hv <= 1 << 18 && B * Hv * chunks <= 1 << 23 && vr <= 1 << 24 &&
                                              kr <= 1 << 24 && T * std::max(kr, vr) <= int64_t(1) << 40;
                            ws_bytes = kan_delta_workspace_size(&d, KAN_PASS_FORWARD);
                            if (!fits) {
                                need(ws_bytes == SIZE_MAX, "too large");
                                continue;
                            }
                            need(ws_bytes < big && (ws_bytes > 0) == (B > 0 && T > 0), "forward workspace");
                            need(kan_delta_forward(&d, at(0), at(1), at(2), at<float>(3), at<float>(4), at<float>(5),
                                                   at<int32_t>(6), at(7), at<float>(8), ws_bytes ? at(9) : nullptr,
                                                   ws_bytes, nullptr) == KAN_OK,
                                 "forward call");
                            ws_bytes = kan_delta_workspace_size(&d, KAN_PASS_BACKWARD);
                            need(ws_bytes < big, "backward workspace");
                            need(kan_delta_backward(&d, at(0), at(1), at(2), at<float>(3), at<float>(4), at<float>(5),
                                                    at<int32_t>(6), at(7), at<float>(8), at(9), at(10), at(11),
                                                    at<float>(12), at<float>(13), at<float>(14),
                                                    ws_bytes ? at(15) : nullptr, ws_bytes, nullptr) == KAN_OK,
                                 "backward call");
                            want += B > 0 ? 2 : 0;
                            if (T == 1 && B > 0) {
                                need(kan_delta_step(&d, B + 5, at(0), at(1), at(2), at<float>(3), at<float>(4),
                                                    at<float>(5), at<int32_t>(6), at(7), nullptr) == KAN_OK,
                                     "step call");
                                ++want;
                            }
                        }
    for (int64_t D : {1, 2, 4, 5, 127, 128, 129, 255, 256, 257, 512, 770, 1024, 1025, 2048, 4096, 4097, 8191, 8192})
        for (int64_t N : {int64_t(0), int64_t(1), int64_t(7), int64_t(8), int64_t(9), int64_t(4999), int64_t(1) << 21,
                          int64_t(1) << 23, int64_t(1) << 25, (int64_t(1) << 25) + 1}) {
            kan_join_desc_t d{N, D, D + 3, D, 2 * D, KAN_BF16, KAN_F32, KAN_BF16, KAN_GATE_SILU,
                              KAN_JOIN_POST | KAN_JOIN_PRE, 1.0f, 1e-6f};
            ws_bytes = kan_join_workspace_size(&d);
            if (N > kan::join_max_rows(D)) {
                need(ws_bytes == SIZE_MAX, "too many rows");
                continue;
            }
            need(ws_bytes < big && (ws_bytes > 0) == (N > 0), "join workspace");
            need(kan_join_forward(&d, at(0), at(1), at(2), at<float>(3), at<float>(4), at(5), at(6), at<float>(7),
                                  nullptr) == KAN_OK,
                 "join forward call");
            need(kan_join_backward(&d, at(0), at(1), at<float>(2), at(3), at(4), at(5), at<float>(6), at<float>(7),
                                   at(8), at(9), at(10), at<float>(11), at<float>(12), ws_bytes ? at(13) : nullptr,
                                   ws_bytes, nullptr) == KAN_OK,
                 "join backward call");
            want += 2;                                 // without rows two fills
        }
    need(launches == want, "a launcher for every call with work");
    printf("ok %ld\n", launches);
    return 0;
}
