// Host-only run of the token-side operators' validation and planning
// (kan_token_api.cpp) under AddressSanitizer and UndefinedBehaviorSanitizer.
// Launcher stubs check what every launcher relies on: plans that cover the
// work, workspaces inside what the caller declared, grids inside the limits of
// a launch.  The driver walks shapes at the edges of the plans' choices and at
// the limits of the descriptions.  Exit status 0 and "ok": everything held.
#include <stdio.h>
#include <stdlib.h>

#include <initializer_list>

#include "kan_token.h"

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
hipError_t launch_embed_fwd(const kan_embed_desc_t& d, const void* ids, const void* E, void* y, hipStream_t) {
    need(ids && E && y && d.N > 0 && d.N * 64 <= kGrid, "embedding forward");    // four rows to a thread of 256
    ++launches;
    return hipSuccess;
}
hipError_t launch_embed_bwd(const kan_embed_desc_t& d, const EmbedPlan& p, const void* ids, const void* dy, float* dE,
                            char* ws, hipStream_t) {
    need(ids && dy && dE && ws && d.N > 0, "embedding backward pointers");
    need(p.chunk > 0 && p.chunks * p.chunk >= d.N && (p.chunks - 1) * p.chunk < d.N, "chunks cover the rows");
    // the ranges end with the one that holds the last token
    int64_t lo = 0, width = 1;
    for (int64_t r = p.ranges - 1;; --r) {
        const int64_t per = kEmbedPerDoubling, k = r < per ? 0 : r / per - 1;
        if (k < kEmbedDoublings) width = int64_t(1) << k, lo = r < per ? r : (per + r % per) << k;
        else width = kEmbedWidth, lo = (per << kEmbedDoublings) + (r - per * (kEmbedDoublings + 1)) * kEmbedWidth;
        break;
    }
    need(p.ranges > 0 && lo < d.V && lo + width >= d.V, "ranges cover the tokens");
    need(p.off_list + (size_t)d.N * 8 <= p.off_start && p.off_start + (size_t)(d.V + 1) * 4 <= p.off_part &&
             p.off_part + (size_t)(p.chunks * 2 * d.D) * 4 <= ws_bytes,
         "workspace carve-outs");
    const int64_t fill = (d.V * d.D + 65535) / 65536;
    need((p.ranges + fill) * 1024 <= kGrid, "listing grid");
    ++launches;
    return hipSuccess;
}
static void recur(const kan_recur_desc_t& d, const RecurPlan& p, const char* ws) {
    need(d.B > 0 && d.D > 0, "recurrence shape");
    need(p.vec == (d.D >= 4 ? 4 : 1) && (p.lanes == 4 || p.lanes == 8 || p.lanes == 16 || p.lanes == 32), "channels of a block");
    need(p.waves >= 1 && p.waves <= kRecurWaves, "waves");
    need((int64_t)p.blocks * p.lanes * p.vec >= d.D && (int64_t)(p.blocks - 1) * p.lanes * p.vec < d.D, "blocks");
    need(p.segs >= 1 && p.segs * p.seg_rows >= d.T && (p.segs == 1 || (p.segs - 1) * p.seg_rows < d.T), "segments");
    need(p.segs == 1 || p.seg_rows % (p.waves * kRecurRows * (64 / p.lanes)) == 0, "segments of whole tiles");
    need(p.segs == 1 ? p.ws == 0 : p.ws >= (size_t)(d.B * p.segs * 2 * d.D) * 4, "runs fit");
    need(p.ws <= ws_bytes && (p.ws == 0 || ws), "workspace");
    need(d.B * p.blocks * p.segs * 64 * p.waves <= kGrid, "recurrence grid");
    ++launches;
}
hipError_t launch_recur_fwd(const kan_recur_desc_t& d, const RecurPlan& p, const RecurArgs& a, char* ws,
                            hipStream_t) {
    need(d.T == 0 || (a.x && a.g && a.out), "forward pointers");
    recur(d, p, ws);
    return hipSuccess;
}
hipError_t launch_recur_bwd(const kan_recur_desc_t& d, const RecurPlan& p, const RecurArgs& a, char* ws,
                            hipStream_t) {
    need((d.T == 0 || (a.x && a.g && a.y && a.dy)) && (a.dx != nullptr) == (a.dg != nullptr), "backward pointers");
    recur(d, p, ws);
    return hipSuccess;
}
hipError_t launch_recur_step(const kan_recur_desc_t& d, int64_t S, const void* x, const void* g, float* state,
                             const int32_t* slots, float* y, hipStream_t) {
    need(d.T == 1 && x && g && y && (S == 0 || state) && (slots || S >= d.B), "step");
    need((d.D + 63) / 64 * d.B * 64 <= kGrid, "step grid");
    ++launches;
    return hipSuccess;
}
hipError_t launch_distill(const kan_distill_desc_t& d, const DistillPlan& p, const DistillArgs& a, char*,
                          hipStream_t) {
    need(d.N > 0 && a.z && a.ids && a.t && a.loss && (a.lse != nullptr) != (a.dz != nullptr), "distillation");
    need(p.ws <= ws_bytes && d.N * 1024 <= kGrid && d.K <= 1024, "distillation plan");
    need(p.parts >= 1 && p.parts <= 64 && p.parts * p.part >= d.V && (p.parts == 1 || p.part % 1024 == 0),
         "parts cover a row");
    need(p.parts == 1 || p.ws >= (size_t)(d.N * p.parts) * 8, "parts' sums fit");
    ++launches;
    return hipSuccess;
}
hipError_t launch_distill_bwd(const kan_distill_desc_t& d, const DistillArgs& a, hipStream_t) {
    need(d.N > 0 && a.z && a.ids && a.t && a.lse_in && a.dloss && a.dz, "distillation backward");
    ++launches;
    return hipSuccess;
}

}  // namespace kan

template <typename T = void>
static T* at(int k) {
    return reinterpret_cast<T*>((uintptr_t)(k + 1) << 50);
}

int main() {
    const size_t big = size_t(1) << 49;
    long want = 0;
    for (int64_t N : {int64_t(0), int64_t(1), int64_t(15), int64_t(16), int64_t(17), int64_t(64), int64_t(4999),
                      int64_t(32768), int64_t(1) << 24})
        for (int64_t V : {int64_t(1), int64_t(15), int64_t(16), int64_t(17), int64_t(31), int64_t(33), int64_t(1000),
                          int64_t(8191), int64_t(8192), int64_t(8193), int64_t(8704), int64_t(8705), int64_t(65536),
                          int64_t(1) << 26})
            for (int64_t D : {int64_t(1), int64_t(3), int64_t(64), int64_t(770), int64_t(4096), int64_t(1) << 23}) {
                kan_embed_desc_t d{N, V, D, KAN_F32, KAN_BF16, KAN_I64, 1.0f};
                ws_bytes = kan_embed_workspace_size(&d);
                if (N > (int64_t(1) << 37) / D || V > (int64_t(1) << 37) / D) {
                    need(ws_bytes == SIZE_MAX, "too many elements");
                    continue;
                }
                need(ws_bytes < big, "embedding workspace");
                need(kan_embed_forward(&d, at(0), at(1), at(2), nullptr) == KAN_OK, "embedding forward call");
                need(kan_embed_backward(&d, at(0), at(1), at<float>(2), at(3), ws_bytes, nullptr) == KAN_OK,
                     "embedding backward call");
                want += N > 0 ? 2 : 1;
            }
    for (int64_t B : {0, 1, 2, 7, 64, 1000, 65536})
        for (int64_t T : {0, 1, 2, 127, 128, 129, 512, 513, 1531, 4096, 65536, 1000003})
            for (int64_t D : {1, 2, 3, 4, 5, 16, 63, 64, 65, 770, 2048, 4096}) {
                kan_recur_desc_t d{B, T, D, 2 * D, 2 * D * T, D, D * T, 2 * D, 2 * D * T, 2 * D, 2 * D * T, 0, 1};
                ws_bytes = kan_recur_workspace_size(&d, KAN_PASS_FORWARD);
                need(ws_bytes < big, "recurrence workspace");
                void* ws = ws_bytes ? at(12) : nullptr;
                need(kan_recur_forward(&d, at(0), at(1), at<float>(2), at<int32_t>(3), at<float>(4), at<float>(5), ws,
                                       ws_bytes, nullptr) == KAN_OK,
                     "recurrence forward call");
                ws_bytes = kan_recur_workspace_size(&d, KAN_PASS_BACKWARD);
                need(ws_bytes < big, "recurrence workspace");
                ws = ws_bytes ? at(12) : nullptr;
                need(kan_recur_backward(&d, at(0), at(1), at<float>(2), at<int32_t>(3), at<float>(4), at<float>(5),
                                        at<float>(6), at(7), reinterpret_cast<char*>(at(7)) + 2 * D, at<float>(9), ws,
                                        ws_bytes, nullptr) == KAN_OK,
                     "recurrence backward call");
                want += B > 0 ? 2 : 0;
            }
    for (int64_t B : {1, 1000, 1 << 22})
        for (int64_t D : {1, 64}) {
            kan_recur_desc_t d{B, 1, D, D, D, D, D, 0, 0, 0, 0, 0, 0};
            need(kan_recur_step(&d, B + 5, at(0), at(1), at<float>(2), at<int32_t>(3), at<float>(4), nullptr) == KAN_OK,
                 "step call");
            ++want;
        }
    for (int64_t N : {0, 1, 16, 4096, 1 << 21})
        for (int64_t V : {int64_t(1), int64_t(1000), int64_t(32003), int64_t(131072), (int64_t(1) << 31) - 4096})
            for (int64_t K : {1, 64, 65, 1024}) {
                kan_distill_desc_t d{N, V, K, V + 3, V, KAN_BF16, KAN_F32, KAN_I32, KAN_F32, 2.0f};
                if (N * V > int64_t(1) << 47) continue;
                ws_bytes = kan_distill_workspace_size(&d);
                need(ws_bytes < big, "distillation workspace");
                void* ws = ws_bytes ? at(12) : nullptr;
                need(kan_distill_forward(&d, at(0), at(1), at(2), at<float>(3), at<float>(4), at<float>(5), ws, ws_bytes,
                                         nullptr) == KAN_OK,
                     "distillation forward call");
                need(kan_distill_step(&d, at(0), at(1), at(2), nullptr, at<float>(4), at(5), ws, ws_bytes, nullptr) ==
                         KAN_OK,
                     "distillation step call");
                need(kan_distill_backward(&d, at(0), at(1), at(2), at<float>(3), at<float>(4), at<float>(5), at(6),
                                          nullptr) == KAN_OK,
                     "distillation backward call");
                want += N > 0 ? 3 : 0;
            }
    need(launches == want, "a launcher for every call with work");
    printf("ok %ld\n", launches);
    return 0;
}
