// Launch plan and kernel launchers of the gated delta rule.
#pragma once

#include "kan_token.h"

namespace kan {

constexpr int kDeltaChunk = 64;      // rows of a chunk
constexpr int64_t kDeltaMaxRow = int64_t(1) << 24;      // stride of rows: 64 of them within 2^32 bytes
constexpr int kDeltaMaxDk = 128;
constexpr int kDeltaMaxDv = 1024;
constexpr int64_t kDeltaMaxHeads = int64_t(1) << 18;    // B Hv
constexpr int64_t kDeltaMaxChunks = int64_t(1) << 23;   // chunks of all heads, B Hv ceil(T / 64)

// What the launches of a call leave each other, in the workspace.  A chunk-head
// is one chunk of one value head: number (b Hv + h) chunks + n.
struct DeltaPlan {
    int dkp, dvp;                    // Dk up to 32, 64 or 128; Dv up to a multiple of 64
    int groups;                      // of 16 state columns, of a scan's block
    int segs, runs, seg_chunks;      // segments of a sequence (1: whole), those whose run is composed, chunks of one
    int64_t chunks, heads;           // of a sequence; B Hv
    int64_t mats;                    // bytes of a chunk-head's matrices
    size_t off_rows;                 // [chunk-head][8][64] float32
    size_t off_mats;                 // [chunk-head][mats]: planes of G, then P (backward: G, G^T, P^T)
    size_t off_w, off_r;             // [chunk-head][64][dvp] float32 (backward)
    size_t off_S, off_dS;            // [chunk-head][dkp][dvp] float32 (backward)
    size_t off_dq, off_dk;           // [B][T][Hv][Dk] float32, where heads share keys (backward)
    size_t off_runs;                 // [segment][head][dkp][dvp + dkp] float32: runs of the segments
    size_t off_starts, off_ends;     // [segment][head][dkp][dvp] float32: their first states; dS at their ends (backward)
    size_t ws;
};
DeltaPlan delta_plan(const kan_delta_desc_t& d, int pass);

struct DeltaArgs {
    const void *q, *k, *v, *dy;
    const float *g, *beta, *h0, *dhT;
    const int32_t* lengths;
    void *y, *dq, *dk, *dv;
    float *hT, *dg, *dbeta, *dh0;
};
hipError_t launch_delta_fwd(const kan_delta_desc_t& d, const DeltaPlan& p, const DeltaArgs& a, char* ws, hipStream_t s);
hipError_t launch_delta_bwd(const kan_delta_desc_t& d, const DeltaPlan& p, const DeltaArgs& a, char* ws, hipStream_t s);
hipError_t launch_delta_step(const kan_delta_desc_t& d, int64_t S, const DeltaArgs& a, float* state,
                             const int32_t* slots, hipStream_t s);

// ---- join ----
constexpr int64_t kJoinMaxD = 8192;
int64_t join_max_rows(int64_t D);
constexpr int kJoinMaxBlocks = 1024; // blocks of a backward pass, each with its own sums for the weights
constexpr int kJoinRows = 4;         // of up to 256 columns that a thread has at a time, where there are many
struct JoinPlan {
    int lanes, vecs;                 // threads of a row, and vectors of four elements that each holds
    int rows;                        // that a thread has at a time (forward)
    unsigned blocks;
    size_t ws;                       // [blocks][2][D] float32 sums of the weights' gradients (backward)
};
JoinPlan join_plan(const kan_join_desc_t& d, int pass);

struct JoinArgs {
    const void *h, *r, *gate, *dy, *dx, *y_in;
    const float *w_post, *w_pre, *stats_in;
    void *y, *x, *dh, *dr, *dgate;
    float *stats, *dw_post, *dw_pre;
};
hipError_t launch_join_fwd(const kan_join_desc_t& d, const JoinPlan& p, const JoinArgs& a, hipStream_t s);
hipError_t launch_join_bwd(const kan_join_desc_t& d, const JoinPlan& p, const JoinArgs& a, char* ws, hipStream_t s);

}  // namespace kan
