// C ABI of the gated delta rule and of the join between blocks: argument
// validation, launch plans and dispatch.  Every check runs before the first
// launch, so a call that fails has enqueued nothing.  No C++ exception leaves
// this file; there is no mutable global state and no device code.
#include <math.h>

#include "kan_checks.h"
#include "kan_delta.h"

namespace kan {

namespace {

// Strided rows [B][T][H][D].
bool strides_ok(const kan_heads_t& s) {
    return stride_ok(s.seq) && s.row >= 0 && s.row <= kDeltaMaxRow && stride_ok(s.head);
}
// Elements from the first to the last of the array, or -1 past 2^60.
int64_t extent4(int64_t B, int64_t T, int64_t H, int64_t D, const kan_heads_t& s) {
    if (B == 0 || T == 0) return 0;
    const __int128 n = (__int128)(B - 1) * s.seq + (__int128)(T - 1) * s.row + (__int128)(H - 1) * s.head + D;
    return n > ((__int128)1 << 60) ? -1 : (int64_t)n;
}
// Whether every dimension lies inside the gaps of another one, so that no two
// rows share an element.
bool distinct(int64_t B, int64_t T, int64_t H, int64_t D, const kan_heads_t& s) {
    struct Dim {
        int64_t n, stride;
    } dims[3] = {{B, s.seq}, {T, s.row}, {H, s.head}};
    if (B == 0 || T == 0) return true;
    std::sort(dims, dims + 3, [](const Dim& a, const Dim& b) { return a.stride < b.stride; });
    __int128 inner = D;
    for (const Dim& m : dims) {
        if (m.n <= 1) continue;
        if (m.stride < inner) return false;
        inner += (__int128)(m.n - 1) * m.stride;
    }
    return true;
}

struct Slice {                       // of an array of gradients
    const void* p;
    kan_heads_t s;
    int64_t H, D;
    Range range(int64_t B, int64_t T, int e) const { return Range{p, (size_t)extent4(B, T, H, D, s) * (size_t)e}; }
};
// Whether two outputs that share a range of memory are slices of one array: some dimensions lie inside
// each slice, whose widths are apart from each other, and the rest, which both have alike, step over both.
bool slices(const Slice& a, const Slice& b, int64_t B, int64_t T, int e) {
    const Slice &lo = reinterpret_cast<uintptr_t>(a.p) < reinterpret_cast<uintptr_t>(b.p) ? a : b, &hi = &lo == &a ? b : a;
    const uintptr_t bytes = reinterpret_cast<uintptr_t>(hi.p) - reinterpret_cast<uintptr_t>(lo.p);
    if (bytes % (unsigned)e) return false;
    const struct {
        int64_t n[2], stride[2];
    } dims[3] = {{{B, B}, {lo.s.seq, hi.s.seq}}, {{T, T}, {lo.s.row, hi.s.row}}, {{lo.H, hi.H}, {lo.s.head, hi.s.head}}};
    for (int inside = 0; inside < 8; ++inside) {       // a bit for each dimension
        __int128 width[2] = {lo.D, hi.D};
        int64_t n[3] = {1, 1, 1}, stride[3] = {};
        bool alike = true;
        for (int x = 0; x < 3; ++x) {
            if (inside >> x & 1) {
                for (int z = 0; z < 2; ++z) width[z] += (__int128)(dims[x].n[z] - 1) * dims[x].stride[z];
            } else {
                n[x] = dims[x].n[0], stride[x] = dims[x].stride[0];
                alike = alike && dims[x].n[1] == n[x] && (n[x] <= 1 || dims[x].stride[1] == stride[x]);
            }
        }
        const __int128 both = bytes / (unsigned)e + width[1];
        if (alike && bytes / (unsigned)e >= width[0] && both <= INT64_MAX &&
            distinct(n[0], n[1], n[2], (int64_t)both, kan_heads_t{stride[0], stride[1], stride[2]}))
            return true;
    }
    return false;
}

int delta_check(const kan_delta_desc_t* d) {
    if (!d) return KAN_ERR_NULL;
    if (!size_ok(d->B, 0) || !size_ok(d->T, 0) || !size_ok(d->Hk, 1) || !size_ok(d->Hv, 1) || d->Hv % d->Hk != 0)
        return KAN_ERR_SHAPE;
    if (d->Dk < 1 || d->Dk > kDeltaMaxDk || d->Dv < 1 || d->Dv > kDeltaMaxDv) return KAN_ERR_SHAPE;
    if (d->B > kDeltaMaxHeads / d->Hv || d->Hv * d->Dv > kDeltaMaxRow) return KAN_ERR_SHAPE;
    const int64_t chunks = (d->T + kDeltaChunk - 1) / kDeltaChunk;
    if (chunks > 0 && d->B * d->Hv > kDeltaMaxChunks / chunks) return KAN_ERR_SHAPE;
    if (!dtype_ok(d->dtype)) return KAN_ERR_DTYPE;
    if (!strides_ok(d->q) || !strides_ok(d->k) || !strides_ok(d->v)) return KAN_ERR_SHAPE;
    if (extent4(d->B, d->T, d->Hk, d->Dk, d->q) < 0 || extent4(d->B, d->T, d->Hk, d->Dk, d->k) < 0 ||
        extent4(d->B, d->T, d->Hv, d->Dv, d->v) < 0)
        return KAN_ERR_SHAPE;
    if ((d->flags & ~KAN_DELTA_UNIT) != 0 || !isfinite(d->scale)) return KAN_ERR_UNSUPPORTED;
    return KAN_OK;
}

int join_check(const kan_join_desc_t* d) {
    if (!d) return KAN_ERR_NULL;
    if (d->D < 1 || d->D > kJoinMaxD || d->N < 0 || d->N > join_max_rows(d->D)) return KAN_ERR_SHAPE;
    if (!dtype_ok(d->dtype) || !dtype_ok(d->res_dtype) || !dtype_ok(d->row_dtype)) return KAN_ERR_DTYPE;
    for (int64_t s : {d->h_row, d->r_row, d->gate_row})
        if (!stride_ok(s)) return KAN_ERR_SHAPE;
    if (extent(d->N, 1, d->D, 0, d->h_row) < 0 || extent(d->N, 1, d->D, 0, d->r_row) < 0 ||
        extent(d->N, 1, d->D, 0, d->gate_row) < 0)
        return KAN_ERR_SHAPE;
    if (d->activation != KAN_GATE_SILU && d->activation != KAN_GATE_SIGMOID) return KAN_ERR_UNSUPPORTED;
    if ((d->flags & ~(KAN_JOIN_POST | KAN_JOIN_PRE)) != 0) return KAN_ERR_UNSUPPORTED;
    if (!isfinite(d->scale) || !isfinite(d->eps) || d->eps < 0.0f) return KAN_ERR_UNSUPPORTED;
    return KAN_OK;
}

}  // namespace

// Whether sequences are cut.  Times in us, of a chunk of a block (a compute unit
// has one at a time) and of what a cut costs once; a run goes through 32 columns of
// the identity for every 32 keys beside those of the values.
static void segments(const kan_delta_desc_t& d, bool back, DeltaPlan& p) {
    const bool f32 = d.dtype == KAN_F32;
    const double pass = f32 ? 5.6 : 4.0, run = f32 ? 4.6 : 3.4, states = f32 ? 4.6 : 4.2, grad = f32 ? 6.5 : 5.5;
    const int64_t tiles = (d.Dv + 31) / 32, wide = tiles + p.dkp / 32;
    auto rounds = [](int64_t blocks) { return (double)((blocks + 255) / 256); };
    double least = 0.0;
    p.segs = 1;
    p.seg_chunks = (int)p.chunks;
    for (int want : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64}) {
        const int64_t each = (p.chunks + want - 1) / want;
        if (want > 1 && each < 4) break;
        const int64_t segs = (p.chunks + each - 1) / std::max<int64_t>(each, 1), runs = segs - (back ? 0 : 1);
        double t = each * rounds(p.heads * segs * tiles) * (back ? states + grad : pass);
        if (segs > 1) {
            t += each * rounds(p.heads * runs * wide) * run + 15.0 + 1.2 * segs;
            if (back) t += each * rounds(p.heads * segs * tiles) * grad + 10.0 + 1.2 * segs;
        }
        if (want == 1 || t < least) {
            least = t;
            p.segs = (int)std::max<int64_t>(segs, 1);
            p.runs = (int)runs;
            p.seg_chunks = (int)each;
        }
    }
    if (p.segs > 1) p.groups = 2;
}

int64_t join_max_rows(int64_t D) { return int64_t(1) << (D > 4096 ? 21 : D > 1024 ? 23 : 25); }

DeltaPlan delta_plan(const kan_delta_desc_t& d, int pass) {
    DeltaPlan p = {};
    const bool back = pass == KAN_PASS_BACKWARD;
    p.dkp = d.Dk <= 32 ? 32 : d.Dk <= 64 ? 64 : 128;
    p.dvp = (int)round_up(d.Dv, 64);
    p.chunks = (d.T + kDeltaChunk - 1) / kDeltaChunk;
    p.heads = d.B * d.Hv;
    p.groups = p.heads * ((d.Dv + 63) / 64) >= 256 ? 4 : 2;
    segments(d, back, p);
    p.mats = (back ? 9 : 6) * int64_t(6 * 64 * 16);    // three planes of each triangular matrix
    size_t off = 0;
    auto take = [&](int64_t bytes) {
        const size_t o = off;
        off += (size_t)round_up(p.heads * p.chunks * bytes, 256);
        return o;
    };
    p.off_rows = take(8 * kDeltaChunk * 4);
    p.off_mats = take(p.mats);
    if (back) {
        p.off_w = take(kDeltaChunk * p.dvp * 4);
        p.off_r = take(kDeltaChunk * p.dvp * 4);
        p.off_S = take((int64_t)p.dkp * p.dvp * 4);
        p.off_dS = take((int64_t)p.dkp * p.dvp * 4);
        if (d.Hv > d.Hk) {
            p.off_dq = take(kDeltaChunk * d.Dk * 4);
            p.off_dk = take(kDeltaChunk * d.Dk * 4);
        }
    }
    if (p.segs > 1) {
        auto segs = [&](int64_t bytes) {
            const size_t o = off;
            off += (size_t)round_up(p.heads * p.segs * bytes, 256);
            return o;
        };
        p.off_runs = segs((int64_t)p.dkp * (p.dvp + p.dkp) * 4);
        p.off_starts = segs((int64_t)p.dkp * p.dvp * 4);
        if (back) p.off_ends = segs((int64_t)p.dkp * p.dvp * 4);
    }
    p.ws = off;
    return p;
}

JoinPlan join_plan(const kan_join_desc_t& d, int pass) {
    JoinPlan p = {};
    const int64_t vectors = (d.D + 3) / 4;
    // A backward pass has nine vectors for each of a row's: at four a thread two waves fill a SIMD's
    // registers, so wide rows go to four waves (4999 x 770 bf16: 48.6 us with one, 31.5 with four).
    const int64_t wave = pass == KAN_PASS_FORWARD ? 256 : 128;
    p.lanes = vectors <= 32 ? 32 : vectors <= wave ? 64 : vectors <= 1024 ? 256 : 1024;
    const int64_t each = (vectors + p.lanes - 1) / p.lanes;
    p.vecs = each <= 1 && (p.lanes <= 64 || pass != KAN_PASS_FORWARD) ? 1 : each <= 2 ? 2 : 4;
    if (p.lanes == 1024) p.vecs = 2;
    const int64_t at_a_time = std::max(1, 256 / p.lanes), blocks = (d.N + at_a_time - 1) / at_a_time;
    p.rows = 1;
    if (pass == KAN_PASS_FORWARD) {
        // still two rounds of blocks on every compute unit
        if (p.vecs == 1 && blocks >= kJoinRows * 4096) p.rows = kJoinRows;
        p.blocks = (unsigned)((blocks + p.rows - 1) / p.rows);
    } else {
        // as many rows to every block
        const int64_t each = std::max<int64_t>((blocks + kJoinMaxBlocks - 1) / kJoinMaxBlocks, 1);
        p.blocks = (unsigned)((blocks + each - 1) / each);
    }
    p.ws = pass == KAN_PASS_FORWARD ? 0 : (size_t)round_up(p.blocks * 2 * d.D * 4, 256);
    return p;
}

}  // namespace kan

using namespace kan;

extern "C" {

size_t kan_delta_workspace_size(const kan_delta_desc_t* desc, int pass) {
    if (delta_check(desc) != KAN_OK || (pass != KAN_PASS_FORWARD && pass != KAN_PASS_BACKWARD)) return SIZE_MAX;
    return desc->B == 0 || desc->T == 0 ? 0 : delta_plan(*desc, pass).ws;
}

int kan_delta_forward(const kan_delta_desc_t* desc, const void* q, const void* k, const void* v, const float* g,
                      const float* beta, const float* h0, const int32_t* lengths, void* y, float* hT, void* ws,
                      size_t ws_bytes, void* stream) {
    int st = delta_check(desc);
    if (st != KAN_OK) return st;
    const kan_delta_desc_t& d = *desc;
    const int e = dtype_bytes(d.dtype);
    if (d.B > 0 && d.T > 0 && (!q || !k || !v || !g || !beta || !y)) return KAN_ERR_NULL;
    if (!aligned(q, e) || !aligned(k, e) || !aligned(v, e) ||
        !all_aligned({g, beta, h0, static_cast<const void*>(lengths), y, hT}, 16))
        return KAN_ERR_ALIGN;
    const size_t need = kan_delta_workspace_size(desc, KAN_PASS_FORWARD);
    if ((st = check_ws(ws, ws_bytes, need)) != KAN_OK) return st;
    const int64_t rows = d.B * d.T * d.Hv, state = d.B * d.Hv * d.Dk * d.Dv;
    const Range outs[] = {{y, (size_t)(rows * d.Dv) * e}, {hT, (size_t)state * 4}, {ws, need}};
    const Range ins[] = {{q, (size_t)extent4(d.B, d.T, d.Hk, d.Dk, d.q) * e},
                         {k, (size_t)extent4(d.B, d.T, d.Hk, d.Dk, d.k) * e},
                         {v, (size_t)extent4(d.B, d.T, d.Hv, d.Dv, d.v) * e},
                         {g, (size_t)rows * 4},
                         {beta, (size_t)rows * 4},
                         {h0, (size_t)state * 4},
                         {lengths, (size_t)d.B * 4}};
    if (any_overlap(outs, ins)) return KAN_ERR_ALIAS;
    if (d.B == 0 || (d.T == 0 && !hT)) return KAN_OK;
    DeltaArgs a = {};
    a.q = q, a.k = k, a.v = v, a.g = g, a.beta = beta, a.h0 = h0, a.lengths = lengths, a.y = y, a.hT = hT;
    (void)hipGetLastError();
    return status_of(launch_delta_fwd(d, delta_plan(d, KAN_PASS_FORWARD), a, static_cast<char*>(ws),
                                      (hipStream_t)stream));
}

int kan_delta_backward(const kan_delta_desc_t* desc, const void* q, const void* k, const void* v, const float* g,
                       const float* beta, const float* h0, const int32_t* lengths, const void* dy, const float* dhT,
                       void* dq, void* dk, void* dv, float* dg, float* dbeta, float* dh0, void* ws, size_t ws_bytes,
                       void* stream) {
    int st = delta_check(desc);
    if (st != KAN_OK) return st;
    const kan_delta_desc_t& d = *desc;
    const int e = dtype_bytes(d.dtype);
    if (d.B > 0 && d.T > 0 && (!q || !k || !v || !g || !beta || !dy || !dq || !dk || !dv || !dg || !dbeta))
        return KAN_ERR_NULL;
    for (const void* p : {q, k, v, static_cast<const void*>(dq), static_cast<const void*>(dk),
                          static_cast<const void*>(dv)})
        if (!aligned(p, e)) return KAN_ERR_ALIGN;
    if (!all_aligned({g, beta, h0, static_cast<const void*>(lengths), dy, dhT, dg, dbeta, dh0}, 16))
        return KAN_ERR_ALIGN;
    const Slice grads[] = {{dq, d.dq, d.Hk, d.Dk}, {dk, d.dk, d.Hk, d.Dk}, {dv, d.dv, d.Hv, d.Dv}};
    for (const Slice& s : grads)
        if (!strides_ok(s.s) || extent4(d.B, d.T, s.H, s.D, s.s) < 0 || !distinct(d.B, d.T, s.H, s.D, s.s))
            return KAN_ERR_SHAPE;
    const size_t need = kan_delta_workspace_size(desc, KAN_PASS_BACKWARD);
    if ((st = check_ws(ws, ws_bytes, need)) != KAN_OK) return st;
    const int64_t rows = d.B * d.T * d.Hv, state = d.B * d.Hv * d.Dk * d.Dv;
    const Range rest[] = {{dg, (size_t)rows * 4}, {dbeta, (size_t)rows * 4}, {dh0, (size_t)state * 4}, {ws, need}};
    const Range ins[] = {{q, (size_t)extent4(d.B, d.T, d.Hk, d.Dk, d.q) * e},
                         {k, (size_t)extent4(d.B, d.T, d.Hk, d.Dk, d.k) * e},
                         {v, (size_t)extent4(d.B, d.T, d.Hv, d.Dv, d.v) * e},
                         {g, (size_t)rows * 4},
                         {beta, (size_t)rows * 4},
                         {h0, (size_t)state * 4},
                         {lengths, (size_t)d.B * 4},
                         {dy, (size_t)(rows * d.Dv) * e},
                         {dhT, (size_t)state * 4}};
    if (any_overlap(rest, ins)) return KAN_ERR_ALIAS;
    for (int x = 0; x < 3; ++x) {
        const Range mine = grads[x].range(d.B, d.T, e);
        for (const Range& r : ins)
            if (overlap(mine, r)) return KAN_ERR_ALIAS;
        for (const Range& r : rest)
            if (overlap(mine, r)) return KAN_ERR_ALIAS;
        for (int z = x + 1; z < 3; ++z)
            if (overlap(mine, grads[z].range(d.B, d.T, e)) && !slices(grads[x], grads[z], d.B, d.T, e))
                return KAN_ERR_ALIAS;
    }
    if (d.B == 0 || (d.T == 0 && !dh0)) return KAN_OK;
    DeltaArgs a = {};
    a.q = q, a.k = k, a.v = v, a.g = g, a.beta = beta, a.h0 = h0, a.lengths = lengths, a.dy = dy, a.dhT = dhT,
    a.dq = dq, a.dk = dk, a.dv = dv, a.dg = dg, a.dbeta = dbeta, a.dh0 = dh0;
    (void)hipGetLastError();
    return status_of(launch_delta_bwd(d, delta_plan(d, KAN_PASS_BACKWARD), a, static_cast<char*>(ws),
                                      (hipStream_t)stream));
}

int kan_delta_step(const kan_delta_desc_t* desc, int64_t S, const void* q, const void* k, const void* v,
                   const float* g, const float* beta, float* state, const int32_t* slots, void* y, void* stream) {
    const int st = delta_check(desc);
    if (st != KAN_OK) return st;
    const kan_delta_desc_t& d = *desc;
    const int e = dtype_bytes(d.dtype);
    if (d.T != 1 || !size_ok(S, 0) || (!slots && S < d.B)) return KAN_ERR_SHAPE;
    if (d.B > 0 && (!q || !k || !v || !g || !beta || !y || (S > 0 && !state))) return KAN_ERR_NULL;
    if (!aligned(q, e) || !aligned(k, e) || !aligned(v, e) ||
        !all_aligned({g, beta, static_cast<const void*>(state), static_cast<const void*>(slots),
                      static_cast<const void*>(y)}, 16))
        return KAN_ERR_ALIGN;
    const int64_t rows = d.B * d.Hv;
    if (S > (int64_t(1) << 58) / (d.Hv * d.Dk * d.Dv)) return KAN_ERR_SHAPE;
    const Range outs[] = {{y, (size_t)(rows * d.Dv) * e}, {state, (size_t)(S * d.Hv * d.Dk * d.Dv) * 4}};
    const Range ins[] = {{q, (size_t)extent4(d.B, 1, d.Hk, d.Dk, d.q) * e},
                         {k, (size_t)extent4(d.B, 1, d.Hk, d.Dk, d.k) * e},
                         {v, (size_t)extent4(d.B, 1, d.Hv, d.Dv, d.v) * e},
                         {g, (size_t)rows * 4},
                         {beta, (size_t)rows * 4},
                         {slots, (size_t)d.B * 4}};
    if (any_overlap(outs, ins)) return KAN_ERR_ALIAS;
    if (d.B == 0) return KAN_OK;
    DeltaArgs a = {};
    a.q = q, a.k = k, a.v = v, a.g = g, a.beta = beta, a.y = y;
    (void)hipGetLastError();
    return status_of(launch_delta_step(d, S, a, state, slots, (hipStream_t)stream));
}

size_t kan_join_workspace_size(const kan_join_desc_t* desc) {
    if (join_check(desc) != KAN_OK) return SIZE_MAX;
    return desc->N == 0 ? 0 : join_plan(*desc, KAN_PASS_BACKWARD).ws;
}

int kan_join_forward(const kan_join_desc_t* desc, const void* h, const void* r, const void* gate,
                     const float* w_post, const float* w_pre, void* y, void* x, float* stats, void* stream) {
    const int st = join_check(desc);
    if (st != KAN_OK) return st;
    const kan_join_desc_t& d = *desc;
    const int e = dtype_bytes(d.dtype), er = dtype_bytes(d.res_dtype), ex = dtype_bytes(d.row_dtype);
    const bool pre = d.flags & KAN_JOIN_PRE;
    if (d.N > 0 && (!h || !y || !stats || (pre && !x))) return KAN_ERR_NULL;
    if (!pre && (x || w_pre)) return KAN_ERR_UNSUPPORTED;
    if (!aligned(h, e) || !aligned(gate, e) || !aligned(r, er) ||
        !all_aligned({w_post, w_pre, static_cast<const void*>(y), static_cast<const void*>(x), stats}, 16))
        return KAN_ERR_ALIGN;
    const Range outs[] = {{y, (size_t)(d.N * d.D) * er}, {x, (size_t)(d.N * d.D) * ex}, {stats, (size_t)d.N * 8}};
    const Range ins[] = {{h, (size_t)extent(d.N, 1, d.D, 0, d.h_row) * e},
                         {r, (size_t)extent(d.N, 1, d.D, 0, d.r_row) * er},
                         {gate, (size_t)extent(d.N, 1, d.D, 0, d.gate_row) * e},
                         {w_post, (size_t)d.D * 4},
                         {w_pre, (size_t)d.D * 4}};
    if (any_overlap(outs, ins)) return KAN_ERR_ALIAS;
    if (d.N == 0) return KAN_OK;
    JoinArgs a = {};
    a.h = h, a.r = r, a.gate = gate, a.w_post = w_post, a.w_pre = w_pre, a.y = y, a.x = x, a.stats = stats;
    (void)hipGetLastError();
    return status_of(launch_join_fwd(d, join_plan(d, KAN_PASS_FORWARD), a, (hipStream_t)stream));
}

int kan_join_backward(const kan_join_desc_t* desc, const void* h, const void* y, const float* stats, const void* dy,
                      const void* dx, const void* gate, const float* w_post, const float* w_pre, void* dh, void* dr,
                      void* dgate, float* dw_post, float* dw_pre, void* ws, size_t ws_bytes, void* stream) {
    int st = join_check(desc);
    if (st != KAN_OK) return st;
    const kan_join_desc_t& d = *desc;
    const int e = dtype_bytes(d.dtype), er = dtype_bytes(d.res_dtype), ex = dtype_bytes(d.row_dtype);
    const bool pre = d.flags & KAN_JOIN_PRE;
    if (d.N > 0 && (!h || !stats || !dh || (dx && !y))) return KAN_ERR_NULL;
    if ((!pre && (dx || w_pre)) || (dgate && !gate) || (dw_post && !w_post) || (dw_pre && !w_pre))
        return KAN_ERR_UNSUPPORTED;
    if (!aligned(h, e) || !aligned(gate, e) ||
        !all_aligned({y, static_cast<const void*>(stats), dy, dx, static_cast<const void*>(w_post),
                      static_cast<const void*>(w_pre), static_cast<const void*>(dh), static_cast<const void*>(dr),
                      static_cast<const void*>(dgate), static_cast<const void*>(dw_post),
                      static_cast<const void*>(dw_pre)}, 16))
        return KAN_ERR_ALIGN;
    const size_t need = dw_post || dw_pre ? kan_join_workspace_size(desc) : 0;
    if ((st = check_ws(ws, ws_bytes, need)) != KAN_OK) return st;
    const size_t n = (size_t)(d.N * d.D);
    const Range outs[] = {{dh, n * e}, {dr, n * er}, {dgate, n * e}, {dw_post, (size_t)d.D * 4},
                          {dw_pre, (size_t)d.D * 4}, {ws, need}};
    const Range ins[] = {{h, (size_t)extent(d.N, 1, d.D, 0, d.h_row) * e},
                         {y, n * er},
                         {stats, (size_t)d.N * 8},
                         {dy, n * er},
                         {dx, n * ex},
                         {gate, (size_t)extent(d.N, 1, d.D, 0, d.gate_row) * e},
                         {w_post, (size_t)d.D * 4},
                         {w_pre, (size_t)d.D * 4}};
    if (any_overlap(outs, ins)) return KAN_ERR_ALIAS;
    hipStream_t s = (hipStream_t)stream;
    (void)hipGetLastError();
    if (d.N == 0) {
        hipError_t err = dw_post ? launch_fill_zero(dw_post, d.D, s) : hipSuccess;
        if (err == hipSuccess && dw_pre) err = launch_fill_zero(dw_pre, d.D, s);
        return status_of(err);
    }
    JoinArgs a = {};
    a.h = h, a.y_in = y, a.stats_in = stats, a.dy = dy, a.dx = dx, a.gate = gate, a.w_post = w_post, a.w_pre = w_pre,
    a.dh = dh, a.dr = dr, a.dgate = dgate, a.dw_post = dw_post, a.dw_pre = dw_pre;
    return status_of(launch_join_bwd(d, join_plan(d, KAN_PASS_BACKWARD), a, static_cast<char*>(ws), s));
}

}  // extern "C"
