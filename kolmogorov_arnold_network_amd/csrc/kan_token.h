// Launch plans and kernel launchers of the token-side operators: embedding,
// gated recurrence, distillation.
#pragma once

#include "kan_internal.h"

namespace kan {

// An array of half the 256 MB cache or more is gone from it before the next
// operator reads it.
constexpr int64_t kStreamBytes = int64_t(128) << 20;

inline int dtype_bytes(int dtype) { return dtype == KAN_F32 ? 4 : 2; }

// ---- embedding ----
// Gradient: the table is cut into ranges of tokens, a block each, that list
// their tokens' rows; the listed rows are summed in chunks.  The ranges are
// kEmbedPerDoubling to a doubling of the token, kEmbedDoublings times, then
// kEmbedWidth tokens each.
constexpr int64_t kEmbedMaxN = int64_t(1) << 24, kEmbedMaxV = int64_t(1) << 26, kEmbedMaxD = int64_t(1) << 23;
constexpr int64_t kEmbedMaxElements = int64_t(1) << 37;     // of the table and of the rows
constexpr int kEmbedPerDoubling = 16, kEmbedDoublings = 9;
constexpr int kEmbedWidth = 1 << kEmbedDoublings;
struct EmbedPlan {
    int chunk;               // listed rows of a chunk
    int64_t ranges, chunks;
    size_t off_list, off_start, off_part, ws;
};
EmbedPlan embed_plan(int64_t N, int64_t V, int64_t D);

hipError_t launch_embed_fwd(const kan_embed_desc_t& d, const void* ids, const void* E, void* y, hipStream_t s);
hipError_t launch_embed_bwd(const kan_embed_desc_t& d, const EmbedPlan& p, const void* ids, const void* dy, float* dE,
                            char* ws, hipStream_t s);

// ---- gated recurrence ----
constexpr int64_t kRecurMaxChannels = int64_t(1) << 28;   // B times D, D rounded up to 64
constexpr int kRecurWaves = 8;       // waves of a block at most
constexpr int kRecurMaxSegs = 256;   // segments of a sequence at most
constexpr int kRecurRows = 4;        // rows of a lane in a tile; a wave has 64 / lanes runs of them
struct RecurPlan {
    int vec, lanes, waves, segs;     // channels of a lane, lanes along the channels, waves of a block, segments
    bool on_lines;                   // rows start on cache lines
    unsigned blocks;                 // channel blocks
    int64_t seg_rows;
    // runs of the segments [B][segs][2][D] float, then marks [B][D] int
    size_t off_marks, ws;
};
RecurPlan recur_plan(const kan_recur_desc_t& d, int pass);

// Channels of lane `cl` of channel block `cb`: `vec` of them from `c` on.  A
// lane whose channels would pass D has the last ones instead; the first
// `before` of those are a channel block's before this one.
struct LaneChannels {
    int64_t c;
    int before;
    __host__ __device__ inline LaneChannels(int64_t cb, int cl, int lanes, int vec, int64_t D) {
        const int64_t first = cb * lanes * vec, own = first + cl * vec;
        c = own < D - vec ? own : D - vec;
        before = c < first ? (int)(first - c) : 0;
    }
};

struct RecurArgs {
    const void *x, *g;
    const float *h0, *y, *dy, *dhT;
    const int32_t* lengths;
    float *out, *hT, *dh0;     // out: y of the forward
    void *dx, *dg;
};
hipError_t launch_recur_fwd(const kan_recur_desc_t& d, const RecurPlan& p, const RecurArgs& a, char* ws, hipStream_t s);
hipError_t launch_recur_bwd(const kan_recur_desc_t& d, const RecurPlan& p, const RecurArgs& a, char* ws, hipStream_t s);
hipError_t launch_recur_step(const kan_recur_desc_t& d, int64_t S, const void* x, const void* g, float* state,
                             const int32_t* slots, float* y, hipStream_t s);

// ---- distillation ----
constexpr int64_t kDistillMaxN = int64_t(1) << 21;
constexpr int kDistillMaxK = 1024;   // teacher logits of a row at most
struct DistillPlan {
    int parts;           // of a row in the step's first launch (1: a block to a row, one launch)
    int64_t part;        // vector elements of a part
    size_t ws;           // maxima and sums of the parts: [N][parts] float2
};
DistillPlan distill_plan(const kan_distill_desc_t& d);

struct DistillArgs {
    const void *z, *ids, *t;
    const float *w, *lse_in, *dloss;
    float *loss, *lse;
    void* dz;
};
hipError_t launch_distill(const kan_distill_desc_t& d, const DistillPlan& p, const DistillArgs& a, char* ws,
                          hipStream_t s);            // forward (a.lse) or step (a.dz)
hipError_t launch_distill_bwd(const kan_distill_desc_t& d, const DistillArgs& a, hipStream_t s);

}  // namespace kan
