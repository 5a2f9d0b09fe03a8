// C ABI of the token-side operators (embedding, gated recurrence,
// distillation): argument validation, launch plans and dispatch.  Every check
// runs before the first launch, so a call that fails has enqueued nothing.
// No C++ exception leaves this file; there is no mutable global state and no
// device code.
#include <math.h>

#include "kan_token.h"

namespace kan {

namespace {

bool dtype_ok(int dtype) { return dtype == KAN_F32 || dtype == KAN_BF16; }
bool index_ok(int t) { return t == KAN_I32 || t == KAN_I64; }
bool size_ok(int64_t n, int64_t least) { return n >= least && n <= kIndexLimit; }
size_t index_bytes(int t) { return t == KAN_I32 ? 4 : 8; }

// Outputs against inputs and against each other.
template <int NO, int NI>
bool any_overlap(const Range (&outs)[NO], const Range (&ins)[NI]) {
    for (int a = 0; a < NO; ++a) {
        for (int b = 0; b < NI; ++b)
            if (overlap(outs[a], ins[b])) return true;
        for (int b = a + 1; b < NO; ++b)
            if (overlap(outs[a], outs[b])) return true;
    }
    return false;
}

template <int NP>
bool all_aligned(const void* const (&ptrs)[NP], uintptr_t a) {
    for (const void* p : ptrs)
        if (p && !aligned(p, a)) return false;
    return true;
}

int check_ws(const void* ws, size_t bytes, size_t need) {
    if (bytes < need) return KAN_ERR_WORKSPACE;
    if (need > 0 && !ws) return KAN_ERR_NULL;
    return ws && !aligned(ws, 256) ? KAN_ERR_ALIGN : KAN_OK;
}

// Strided rows [B][T][D].  A stride past 2^40 elements is refused, so that
// extents fit 64 bits with any B and T.
constexpr int64_t kStrideLimit = int64_t(1) << 40;
bool stride_ok(int64_t s) { return s >= 0 && s <= kStrideLimit; }
// Elements from the first to the last of the array, or -1 past 2^60.
int64_t extent(int64_t B, int64_t T, int64_t D, int64_t row, int64_t seq) {
    if (B == 0 || T == 0) return 0;
    const __int128 n = (__int128)(B - 1) * seq + (__int128)(T - 1) * row + D;
    return n > ((__int128)1 << 60) ? -1 : (int64_t)n;
}
// The least distance between the starts of two rows: 0 where rows of the
// array may interleave in another way than one stride inside the other.
int64_t row_distance(int64_t B, int64_t T, int64_t row, int64_t seq) {
    if (B <= 1 && T <= 1) return INT64_MAX;
    if (B <= 1) return row;
    if (T <= 1) return seq;
    const __int128 in_rows = (__int128)seq - (__int128)(T - 1) * row;   // sequences apart
    const __int128 in_seqs = (__int128)row - (__int128)(B - 1) * seq;   // sequences interleaved
    if (in_rows > 0) return (int64_t)std::min<__int128>(row, in_rows);
    if (in_seqs > 0) return (int64_t)std::min<__int128>(seq, in_seqs);
    return 0;
}

int embed_check(const kan_embed_desc_t* d) {
    if (!d) return KAN_ERR_NULL;
    if (d->N < 0 || d->N > kEmbedMaxN || d->V < 1 || d->V > kEmbedMaxV || d->D < 1 || d->D > kEmbedMaxD)
        return KAN_ERR_SHAPE;
    if (d->N > kEmbedMaxElements / d->D || d->V > kEmbedMaxElements / d->D) return KAN_ERR_SHAPE;
    if (!dtype_ok(d->dtype) || !dtype_ok(d->row_dtype) || !index_ok(d->id_dtype)) return KAN_ERR_DTYPE;
    if (!isfinite(d->scale)) return KAN_ERR_UNSUPPORTED;
    return KAN_OK;
}

int recur_check(const kan_recur_desc_t* d) {
    if (!d) return KAN_ERR_NULL;
    if (!size_ok(d->B, 0) || !size_ok(d->T, 0) || !size_ok(d->D, 1)) return KAN_ERR_SHAPE;
    if (d->B > kRecurMaxChannels / round_up(d->D, 64)) return KAN_ERR_SHAPE;
    if (d->B > 0 && d->T > (int64_t(1) << 60) / d->B / d->D) return KAN_ERR_SHAPE;
    if (!dtype_ok(d->dtype) || !dtype_ok(d->grad_dtype)) return KAN_ERR_DTYPE;
    for (int64_t s : {d->x_row, d->x_seq, d->g_row, d->g_seq, d->dx_row, d->dx_seq, d->dg_row, d->dg_seq})
        if (!stride_ok(s)) return KAN_ERR_SHAPE;
    if (extent(d->B, d->T, d->D, d->x_row, d->x_seq) < 0 || extent(d->B, d->T, d->D, d->g_row, d->g_seq) < 0)
        return KAN_ERR_SHAPE;
    return KAN_OK;
}

int distill_check(const kan_distill_desc_t* d, bool grad) {
    if (!d) return KAN_ERR_NULL;
    if (d->N < 0 || d->N > kDistillMaxN || !size_ok(d->V, 1) || d->K < 1 || d->K > kDistillMaxK) return KAN_ERR_SHAPE;
    if (d->z_row < d->V || !stride_ok(d->z_row)) return KAN_ERR_SHAPE;
    if (grad && (d->dz_row < d->V || !stride_ok(d->dz_row))) return KAN_ERR_SHAPE;
    if (extent(d->N, 1, d->V, 0, d->z_row) < 0 || (grad && extent(d->N, 1, d->V, 0, d->dz_row) < 0))
        return KAN_ERR_SHAPE;
    if (!dtype_ok(d->dtype) || !dtype_ok(d->teacher_dtype) || !index_ok(d->id_dtype)) return KAN_ERR_DTYPE;
    if (grad && !dtype_ok(d->grad_dtype)) return KAN_ERR_DTYPE;
    if (!isfinite(d->tau) || !(d->tau > 0.0f)) return KAN_ERR_UNSUPPORTED;
    return KAN_OK;
}

// Pointer checks shared by the distillation entry points; the ranges of their
// inputs in `in`.
int distill_inputs(const kan_distill_desc_t& d, const void* z, const void* ids, const void* t, const float* w,
                   Range (&in)[6]) {
    if (d.N > 0 && (!z || !ids || !t)) return KAN_ERR_NULL;
    if (!aligned(z, dtype_bytes(d.dtype)) || !all_aligned({ids, t, w}, 16)) return KAN_ERR_ALIGN;
    in[0] = Range{z, (size_t)extent(d.N, 1, d.V, 0, d.z_row) * dtype_bytes(d.dtype)};
    in[1] = Range{ids, (size_t)(d.N * d.K) * index_bytes(d.id_dtype)};
    in[2] = Range{t, (size_t)(d.N * d.K) * dtype_bytes(d.teacher_dtype)};
    in[3] = Range{w, (size_t)d.N * 4};
    in[4] = in[5] = Range{nullptr, 0};
    return KAN_OK;
}

}  // namespace

EmbedPlan embed_plan(int64_t N, int64_t V, int64_t D) {
    EmbedPlan p;
    // as the ranges are numbered on the device
    constexpr int64_t per = kEmbedPerDoubling, wide = per << kEmbedDoublings;
    p.ranges = std::min(V, per);
    for (int k = 0; k < kEmbedDoublings && V > per << k; ++k)
        p.ranges += std::min(per, (V - (per << k) + (int64_t(1) << k) - 1) >> k);
    if (V > wide) p.ranges += (V - wide + kEmbedWidth - 1) / kEmbedWidth;
    // Long chunks leave fewer tokens to join, short ones make more waves (each
    // sums a chunk in 256 columns): 64 rows where that still makes 4096 waves,
    // else 16 (4999 rows of 770: 27.8 us with 32, 25.3 with 16).
    p.chunk = N / 64 * ((D + 255) / 256) >= 4096 ? 64 : 16;
    p.chunks = (N + p.chunk - 1) / p.chunk;
    size_t off = 0;
    auto take = [&](int64_t bytes) {
        const size_t o = off;
        off += (size_t)round_up(bytes, 256);
        return o;
    };
    p.off_list = take(N * 8);
    p.off_start = take((V + 1) * 4);
    p.off_part = take(p.chunks * 2 * D * 4);
    p.ws = off;
    return p;
}

RecurPlan recur_plan(const kan_recur_desc_t& d, int pass) {
    // Time is counted in tiles of 128 rows by 64 channels, of which 256, one for
    // each compute unit, take about as long as their memory traffic.  A launch
    // takes as many as the longest block has, 1.4 times that where a unit holds
    // two blocks, and no less than its traffic.  Blocks with fewer lanes along
    // the channels make more and shorter columns, but touch more cache lines
    // for their bytes, above all where rows do not start on a line; measured,
    // time goes with the lines to the power 0.75 or so (8 x 4096 x 2048 bf16
    // forward: 106 us with 16 lanes, 126 with 8; 70 x 1531 x 770 bf16 backward:
    // 461 with 32, 529 with 16, 364 with 16 at 768 channels).  Segments read a
    // little twice and take two launches more (1 x 65536 x 1024 float32 forward:
    // 564 us whole with 4 lanes, 172 in segments).  Of 19 shapes between 1 x 2048 x
    // 1024 and 8 x 1024 x 768, timed with each of the plans below, the chosen one
    // is the best or up to 13% over it (7 x 1531 x 770 bf16, lengths drawn:
    // backward 62 us, 69 whole with 8 lanes; forward 38, 33 whole with 8 lanes).
    constexpr int64_t kCUs = 256;
    const bool forward = pass == KAN_PASS_FORWARD;
    RecurPlan p;
    p.vec = d.D >= 4 ? 4 : 1;
    const int es = dtype_bytes(d.dtype);
    p.on_lines = (d.D * 4) % 128 == 0 && (d.x_row * es) % 128 == 0 && (d.g_row * es) % 128 == 0;
    if (!forward)
        p.on_lines = p.on_lines && (d.dx_row * dtype_bytes(d.grad_dtype)) % 128 == 0 &&
                     (d.dg_row * dtype_bytes(d.grad_dtype)) % 128 == 0;
    const int64_t T = std::max<int64_t>(d.T, 1);
    // cache lines that a block's row touches in its arrays, over the least that
    // its bytes need
    auto lines = [&](int lanes) {
        double touched = 0, least = 0;
        auto array = [&](int bytes, int count) {
            const double own = lanes * p.vec * bytes / 128.0;
            touched += count * (p.on_lines ? std::max(own, 1.0) : own + 1.0);
            least += count * own;
        };
        array(es, 2);
        array(4, forward ? 1 : 2);
        if (!forward) array(dtype_bytes(d.grad_dtype), 2);
        return pow(touched / least, 0.75);
    };
    double least = -1.0;
    auto weigh = [&](int lanes, int64_t want) {        // want: blocks, in segments (0: whole)
        const int64_t tile = kRecurWaves * kRecurRows * (64 / lanes);
        const int64_t blocks = (d.D + lanes * p.vec - 1) / (lanes * p.vec), have = std::max<int64_t>(1, d.B * blocks);
        int64_t segs = std::min<int64_t>(std::min<int64_t>(kRecurMaxSegs, want / have), T / tile);
        if (want > 0 && segs < 2) return;
        const int64_t rows = segs > 1 ? round_up((T + segs - 1) / segs, tile) : T;
        segs = (T + rows - 1) / rows;
        const int64_t n = have * segs;
        const double most = n <= kCUs ? 1.0 : 1.4 * (double)((n + 2 * kCUs - 1) / (2 * kCUs));
        const double tiles = (double)((rows + tile - 1) / tile);
        const double traffic = (double)d.B * (double)T * (double)d.D / (128.0 * 64.0 * kCUs);
        const bool cut = segs > 1;
        const double est = std::max(most * tiles, traffic) * lines(lanes) * (cut ? 1.1 : 1.0) + (cut ? 3.0 : 0.0);
        if (least >= 0.0 && est >= least) return;
        least = est;
        p.lanes = lanes;
        p.segs = (int)segs;
        p.seg_rows = rows;
        p.blocks = (unsigned)blocks;
    };
    if (p.vec == 1) {
        weigh(4, 0);
        weigh(4, kCUs);
    } else {
        for (int lanes : {32, 16, 8, 4}) weigh(lanes, 0);
        for (int lanes : {32, 16, 8}) weigh(lanes, kCUs), weigh(lanes, 2 * kCUs);
    }
    const int wave_rows = kRecurRows * (64 / p.lanes);
    p.waves = 1;
    while (p.waves < kRecurWaves && p.waves * wave_rows < p.seg_rows) p.waves *= 2;
    p.off_marks = p.segs > 1 ? (size_t)round_up(d.B * p.segs * 2 * d.D * 4, 256) : 0;
    p.ws = p.segs > 1 ? p.off_marks + (size_t)round_up(d.B * d.D * 4, 256) : 0;
    return p;
}

DistillPlan distill_plan(const kan_distill_desc_t& d) {
    // A step of few long rows is cut over blocks: its maxima and sums in one
    // launch, the gradient in a second.  With a block to a row its time is one
    // compute unit's arithmetic.  Whole and cut, us: one row of 131072 logits 19.8
    // and 13.8 (bf16 22.6, 13.8), 64 rows 31.0 and 25.4 (26.6, 17.2); 64 rows of
    // 98304 24.4 and 21.3 (22.2, 16.3); one row of 65536 11.5 and 14.2 (13.9, 13.9).
    // With more rows than 64 the gain ends, at 96 in float32 (34.9, 33.9; 98304
    // logits: 26.4, 29.3) and between 128 and 192 in bf16.
    DistillPlan p{1, d.V, 0};
    if (d.N > 0 && d.N <= 64 && d.V >= 98304) {
        const int64_t want = std::min<int64_t>(std::min<int64_t>(64, 512 / d.N), d.V / 4096);
        p.part = round_up((d.V + want - 1) / want, 1024);
        p.parts = (int)((d.V + p.part - 1) / p.part);
        if (p.parts > 1) p.ws = (size_t)round_up(d.N * p.parts * 8, 256);
    }
    return p;
}

}  // namespace kan

using namespace kan;

extern "C" {

size_t kan_embed_workspace_size(const kan_embed_desc_t* desc) {
    if (embed_check(desc) != KAN_OK) return SIZE_MAX;
    return desc->N == 0 ? 0 : embed_plan(desc->N, desc->V, desc->D).ws;
}

int kan_embed_forward(const kan_embed_desc_t* desc, const void* ids, const void* E, void* y, void* stream) {
    const int st = embed_check(desc);
    if (st != KAN_OK) return st;
    const int64_t N = desc->N, D = desc->D;
    if (!E || (N > 0 && (!ids || !y))) return KAN_ERR_NULL;
    if (!all_aligned({ids, E, static_cast<const void*>(y)}, 16)) return KAN_ERR_ALIGN;
    const Range outs[] = {{y, (size_t)(N * D) * dtype_bytes(desc->row_dtype)}};
    const Range ins[] = {{ids, (size_t)N * index_bytes(desc->id_dtype)},
                         {E, (size_t)(desc->V * D) * dtype_bytes(desc->dtype)}};
    if (any_overlap(outs, ins)) return KAN_ERR_ALIAS;
    if (N == 0) return KAN_OK;
    (void)hipGetLastError();
    return status_of(launch_embed_fwd(*desc, ids, E, y, (hipStream_t)stream));
}

int kan_embed_backward(const kan_embed_desc_t* desc, const void* ids, const void* dy, float* dE, void* ws,
                       size_t ws_bytes, void* stream) {
    int st = embed_check(desc);
    if (st != KAN_OK) return st;
    const int64_t N = desc->N, V = desc->V, D = desc->D;
    if (!dE || (N > 0 && (!ids || !dy))) return KAN_ERR_NULL;
    if (!all_aligned({ids, dy, static_cast<const void*>(dE)}, 16)) return KAN_ERR_ALIGN;
    const size_t need = kan_embed_workspace_size(desc);
    if ((st = check_ws(ws, ws_bytes, need)) != KAN_OK) return st;
    const Range outs[] = {{dE, (size_t)(V * D) * 4}, {ws, need}};
    const Range ins[] = {{ids, (size_t)N * index_bytes(desc->id_dtype)},
                         {dy, (size_t)(N * D) * dtype_bytes(desc->row_dtype)}};
    if (any_overlap(outs, ins)) return KAN_ERR_ALIAS;
    hipStream_t s = (hipStream_t)stream;
    (void)hipGetLastError();
    if (N == 0) return status_of(launch_fill_zero(dE, V * D, s));
    return status_of(launch_embed_bwd(*desc, embed_plan(N, V, D), ids, dy, dE, static_cast<char*>(ws), s));
}

size_t kan_recur_workspace_size(const kan_recur_desc_t* desc, int pass) {
    if (recur_check(desc) != KAN_OK || (pass != KAN_PASS_FORWARD && pass != KAN_PASS_BACKWARD)) return SIZE_MAX;
    return desc->B == 0 || desc->T == 0 ? 0 : recur_plan(*desc, pass).ws;
}

int kan_recur_forward(const kan_recur_desc_t* desc, const void* x, const void* g, const float* h0,
                      const int32_t* lengths, float* y, float* hT, void* ws, size_t ws_bytes, void* stream) {
    int st = recur_check(desc);
    if (st != KAN_OK) return st;
    const int64_t B = desc->B, T = desc->T, D = desc->D;
    const int es = dtype_bytes(desc->dtype);
    if (B > 0 && T > 0 && (!x || !g || !y)) return KAN_ERR_NULL;
    if (!aligned(x, es) || !aligned(g, es) || !all_aligned({h0, lengths, y, hT}, 16)) return KAN_ERR_ALIGN;
    const size_t need = kan_recur_workspace_size(desc, KAN_PASS_FORWARD);
    if ((st = check_ws(ws, ws_bytes, need)) != KAN_OK) return st;
    const Range outs[] = {{y, (size_t)(B * T * D) * 4}, {hT, (size_t)(B * D) * 4}, {ws, need}};
    const Range ins[] = {{x, (size_t)extent(B, T, D, desc->x_row, desc->x_seq) * es},
                         {g, (size_t)extent(B, T, D, desc->g_row, desc->g_seq) * es},
                         {h0, (size_t)(B * D) * 4},
                         {lengths, (size_t)B * 4}};
    if (any_overlap(outs, ins)) return KAN_ERR_ALIAS;
    if (B == 0 || (T == 0 && !hT)) return KAN_OK;
    RecurArgs a = {};
    a.x = x, a.g = g, a.h0 = h0, a.lengths = lengths, a.out = y, a.hT = hT;
    (void)hipGetLastError();
    return status_of(launch_recur_fwd(*desc, recur_plan(*desc, KAN_PASS_FORWARD), a, static_cast<char*>(ws),
                                      (hipStream_t)stream));
}

int kan_recur_backward(const kan_recur_desc_t* desc, const void* x, const void* g, const float* h0,
                       const int32_t* lengths, const float* y, const float* dy, const float* dhT, void* dx, void* dg,
                       float* dh0, void* ws, size_t ws_bytes, void* stream) {
    int st = recur_check(desc);
    if (st != KAN_OK) return st;
    const int64_t B = desc->B, T = desc->T, D = desc->D;
    const int es = dtype_bytes(desc->dtype), eg = dtype_bytes(desc->grad_dtype);
    if ((dx != nullptr) != (dg != nullptr)) return KAN_ERR_NULL;
    if (B > 0 && T > 0 && (!x || !g || !y || !dy)) return KAN_ERR_NULL;
    if (!aligned(x, es) || !aligned(g, es) || !aligned(dx, eg) || !aligned(dg, eg) ||
        !all_aligned({h0, lengths, y, dy, dhT, static_cast<const float*>(dh0)}, 16))
        return KAN_ERR_ALIGN;
    const int64_t ndx = extent(B, T, D, desc->dx_row, desc->dx_seq), ndg = extent(B, T, D, desc->dg_row, desc->dg_seq);
    if (dx && (ndx < 0 || ndg < 0)) return KAN_ERR_SHAPE;
    const size_t need = kan_recur_workspace_size(desc, KAN_PASS_BACKWARD);
    if ((st = check_ws(ws, ws_bytes, need)) != KAN_OK) return st;
    const Range rdx{dx, (size_t)ndx * eg}, rdg{dg, (size_t)ndg * eg};
    const Range rest[] = {{dh0, (size_t)(B * D) * 4}, {ws, need}};
    const Range ins[] = {{x, (size_t)extent(B, T, D, desc->x_row, desc->x_seq) * es},
                         {g, (size_t)extent(B, T, D, desc->g_row, desc->g_seq) * es},
                         {h0, (size_t)(B * D) * 4},
                         {lengths, (size_t)B * 4},
                         {y, (size_t)(B * T * D) * 4},
                         {dy, (size_t)(B * T * D) * 4},
                         {dhT, (size_t)(B * D) * 4}};
    if (any_overlap(rest, ins)) return KAN_ERR_ALIAS;
    if (dx && B > 0 && T > 0) {
        const Range grads[] = {rdx, rdg};
        for (const Range& r : grads) {
            for (const Range& q : ins)
                if (overlap(r, q)) return KAN_ERR_ALIAS;
            for (const Range& q : rest)
                if (overlap(r, q)) return KAN_ERR_ALIAS;
        }
        const int64_t mx = row_distance(B, T, desc->dx_row, desc->dx_seq);
        const int64_t mg = row_distance(B, T, desc->dg_row, desc->dg_seq);
        if (mx < D || mg < D) return KAN_ERR_SHAPE;
        if (overlap(rdx, rdg)) {
            // two halves of one array: the same strides, and every row of one
            // inside the gap between two rows of the other
            const uintptr_t px = reinterpret_cast<uintptr_t>(dx), pg = reinterpret_cast<uintptr_t>(dg);
            const int64_t apart = (int64_t)((px < pg ? pg - px : px - pg) / (unsigned)eg);
            if (desc->dx_row != desc->dg_row || desc->dx_seq != desc->dg_seq || apart < D || mx - D < apart)
                return KAN_ERR_ALIAS;
        }
    }
    if (B == 0 || (!dx && !dh0) || (T == 0 && !dh0)) return KAN_OK;
    RecurArgs a = {};
    a.x = x, a.g = g, a.h0 = h0, a.lengths = lengths, a.y = y, a.dy = dy, a.dhT = dhT, a.dx = dx, a.dg = dg,
    a.dh0 = dh0;
    (void)hipGetLastError();
    return status_of(launch_recur_bwd(*desc, recur_plan(*desc, KAN_PASS_BACKWARD), a, static_cast<char*>(ws),
                                      (hipStream_t)stream));
}

int kan_recur_step(const kan_recur_desc_t* desc, int64_t S, const void* x, const void* g, float* state,
                   const int32_t* slots, float* y, void* stream) {
    const int st = recur_check(desc);
    if (st != KAN_OK) return st;
    const int64_t B = desc->B, D = desc->D;
    const int es = dtype_bytes(desc->dtype);
    if (desc->T != 1 || !size_ok(S, 0) || (!slots && S < B)) return KAN_ERR_SHAPE;
    if (B > 0 && (!x || !g || !y || (S > 0 && !state))) return KAN_ERR_NULL;
    if (!aligned(x, es) || !aligned(g, es) || !all_aligned({static_cast<const void*>(state), slots, y}, 16))
        return KAN_ERR_ALIGN;
    const Range outs[] = {{y, (size_t)(B * D) * 4}, {state, (size_t)(S * D) * 4}};
    const Range ins[] = {{x, (size_t)extent(B, 1, D, desc->x_row, desc->x_seq) * es},
                         {g, (size_t)extent(B, 1, D, desc->g_row, desc->g_seq) * es},
                         {slots, (size_t)B * 4}};
    if (any_overlap(outs, ins)) return KAN_ERR_ALIAS;
    if (B == 0) return KAN_OK;
    (void)hipGetLastError();
    return status_of(launch_recur_step(*desc, S, x, g, state, slots, y, (hipStream_t)stream));
}

size_t kan_distill_workspace_size(const kan_distill_desc_t* desc) {
    if (distill_check(desc, false) != KAN_OK) return SIZE_MAX;
    return desc->N == 0 ? 0 : distill_plan(*desc).ws;
}

int kan_distill_forward(const kan_distill_desc_t* desc, const void* z, const void* ids, const void* t,
                        const float* w, float* loss, float* lse, void* ws, size_t ws_bytes, void* stream) {
    int st = distill_check(desc, false);
    if (st != KAN_OK) return st;
    Range in[6];
    if ((st = distill_inputs(*desc, z, ids, t, w, in)) != KAN_OK) return st;
    if (desc->N > 0 && (!loss || !lse)) return KAN_ERR_NULL;
    if (!all_aligned({loss, lse}, 16)) return KAN_ERR_ALIGN;
    if ((st = check_ws(ws, ws_bytes, 0)) != KAN_OK) return st;      // only the step's rows are cut
    const Range outs[] = {{loss, (size_t)desc->N * 4}, {lse, (size_t)desc->N * 4}};
    if (any_overlap(outs, in)) return KAN_ERR_ALIAS;
    if (desc->N == 0) return KAN_OK;
    DistillArgs a = {};
    a.z = z, a.ids = ids, a.t = t, a.w = w, a.loss = loss, a.lse = lse;
    (void)hipGetLastError();
    return status_of(launch_distill(*desc, DistillPlan{1, desc->V, 0}, a, nullptr, (hipStream_t)stream));
}

int kan_distill_backward(const kan_distill_desc_t* desc, const void* z, const void* ids, const void* t,
                         const float* w, const float* lse, const float* dloss, void* dz, void* stream) {
    int st = distill_check(desc, true);
    if (st != KAN_OK) return st;
    Range in[6];
    if ((st = distill_inputs(*desc, z, ids, t, w, in)) != KAN_OK) return st;
    if (desc->N > 0 && (!lse || !dloss || !dz)) return KAN_ERR_NULL;
    if (!all_aligned({lse, dloss}, 16) || !aligned(dz, dtype_bytes(desc->grad_dtype))) return KAN_ERR_ALIGN;
    in[4] = Range{lse, (size_t)desc->N * 4};
    in[5] = Range{dloss, (size_t)desc->N * 4};
    const Range outs[] = {{dz, (size_t)extent(desc->N, 1, desc->V, 0, desc->dz_row) * dtype_bytes(desc->grad_dtype)}};
    if (any_overlap(outs, in)) return KAN_ERR_ALIAS;
    if (desc->N == 0) return KAN_OK;
    DistillArgs a = {};
    a.z = z, a.ids = ids, a.t = t, a.w = w, a.lse_in = lse, a.dloss = dloss, a.dz = dz;
    (void)hipGetLastError();
    return status_of(launch_distill_bwd(*desc, a, (hipStream_t)stream));
}

int kan_distill_step(const kan_distill_desc_t* desc, const void* z, const void* ids, const void* t, const float* w,
                     float* loss, void* dz, void* ws, size_t ws_bytes, void* stream) {
    int st = distill_check(desc, true);
    if (st != KAN_OK) return st;
    Range in[6];
    if ((st = distill_inputs(*desc, z, ids, t, w, in)) != KAN_OK) return st;
    if (desc->N > 0 && (!loss || !dz)) return KAN_ERR_NULL;
    if (!aligned(loss, 16) || !aligned(dz, dtype_bytes(desc->grad_dtype))) return KAN_ERR_ALIGN;
    const size_t need = kan_distill_workspace_size(desc);
    if ((st = check_ws(ws, ws_bytes, need)) != KAN_OK) return st;
    const Range outs[] = {{loss, (size_t)desc->N * 4},
                          {dz, (size_t)extent(desc->N, 1, desc->V, 0, desc->dz_row) * dtype_bytes(desc->grad_dtype)},
                          {ws, need}};
    if (any_overlap(outs, in)) return KAN_ERR_ALIAS;
    if (desc->N == 0) return KAN_OK;
    DistillArgs a = {};
    a.z = z, a.ids = ids, a.t = t, a.w = w, a.loss = loss, a.dz = dz;
    (void)hipGetLastError();
    return status_of(launch_distill(*desc, distill_plan(*desc), a, static_cast<char*>(ws), (hipStream_t)stream));
}

}  // extern "C"
