// Gated linear recurrence over the rows of a sequence, each channel on its own
// (gfx950):
//
//     u_t = sigmoid(-g_t),  h_t = h_{t-1} + u_t (x_t - h_{t-1})
//
// its backward pass, and its single-row step on a pool of states.
//
// Backward, with c_t = f_t del_t the gradient that row t hands to row t - 1
// (c_len = dhT):
//
//     del_t = dy_t + c_{t+1},  dx_t = u_t del_t,
//     dg_t  = f_t (h_{t-1} - x_t) dx_t,  dh0 = c_0.
//
// Both shares are computed relative to their own size: a share that rounds to 1
// has lost the digits of the other one, which decide how long a memory is (f
// near 1) or how much of a large state is left (u near 1).  Where a state goes
// on from tile to tile, or from call to call in the single step, it changes by
// the smaller share alone, h + u (x - h) or x + f (h - x).
//
// A run of steps is h -> L h + b with L = prod f, kept like a gate: by the
// smaller of L and U = 1 - L.  Two runs compose to one (the earlier first):
// L = L1 L2, U = U1 + U2 L1, b = b2 + L2 b1.  A block takes 16 to 128 channels
// of a sequence and walks along it in tiles, each read once: lanes hold four
// channels of four consecutive rows in registers and compose them, the runs of
// a wave's lanes and of the block's 8 waves are scanned, and every row's state
// follows from its lane's start.  The next tile's loads are issued before the
// scan.  (Eight rows to a lane and 16 waves to a block took 1.2 and 1.1 times as
// long: fewer blocks to a compute unit.)  Where the sequences have too few
// channels to fill the GPU they are cut into segments, a block each: a first
// launch composes every segment's run, from as many of its rows as still count
// at its end, and the second starts each segment from the runs before it.
//
// Memory traffic bounds it: 8 x 4096 x 2048, bf16 forward 104 us (537 MB, 5.2
// TB/s), float32 backward 316 us (1.61 GB, 5.1 TB/s), 1 x 65536 x 1024 float32
// forward 166 us (805 MB, 4.9 TB/s: 13 for the segments' runs, 146 for the rows, 4
// for the launch that looks at marks), where a copy runs at 5.0 TB/s.  The
// arithmetic (two transcendentals and about 25 operations an element forward)
// keeps the vector units busy for half of that.
#include <type_traits>

#include "kan_token.h"
#include "kan_vec.h"

namespace kan {

namespace {

// The shares of x and of the state, u = sigmoid(-g) and f = sigmoid(g).  The
// smaller one is within (1.3 |g| + 12) 2^-24 of its own size: exp's argument,
// |g| log2 e, rounds.  The larger one is within a few ulp.
struct Shares {
    float u, f;
    __device__ __forceinline__ static Shares of(float g) {
        const float v = __expf(-fabsf(g)), most = __builtin_amdgcn_rcpf(1.0f + v), least = v * most;
        return g < 0.0f ? Shares{most, least} : Shares{least, most};
    }
    __device__ __forceinline__ static Shares idle() { return Shares{0.0f, 1.0f}; }     // the state stays
};

// The same as one word: the smaller of the two, with the sign bit set where it
// is f.  The larger one is 1 less it, and a state changes by it without the
// rounding of the larger one, which would add up over a long memory.
struct Gate {
    float e;
    __device__ __forceinline__ static Gate of(float g) {
        const float v = __expf(-fabsf(g));
        return Gate{__builtin_copysignf(v * __builtin_amdgcn_rcpf(1.0f + v), g)};
    }
    __device__ __forceinline__ static Gate idle() { return Gate{0.0f}; }
    __device__ __forceinline__ static Gate of(Shares q) { return Gate{q.u < 0.5f ? q.u : -q.f}; }
    __device__ __forceinline__ bool keep() const { return (int)__float_as_uint(e) >= 0; }
    __device__ __forceinline__ Shares shares() const {
        return Shares{keep() ? e : 1.0f + e, keep() ? 1.0f - e : -e};
    }
    // f h + u x; as it stands where the difference overflows or has an infinity in it
    __device__ __forceinline__ float step(float h, float x) const {
        const float a = keep() ? h : x, b = keep() ? x : h;
        const float n = __builtin_fmaf(fabsf(e), b - a, a);
        const Shares q = shares();
        return __builtin_isfinite(n) ? n : __builtin_fmaf(q.f, h, q.u * x);
    }
    // what is left of h: f h, for a finite h (an infinity may become NaN)
    __device__ __forceinline__ float of_state(float h) const { return __builtin_fmaf(-e, h, keep() ? h : 0.0f); }
};

constexpr int RW = kRecurWaves;    // waves of a block at most

__device__ __forceinline__ int64_t length_of(const int32_t* lengths, int64_t b, int64_t T) {
    return lengths ? min(max((int64_t)lengths[b], (int64_t)0), T) : T;
}

constexpr int kRunsLanes(int vec) { return vec == 1 ? 4 : 16; }    // of the launch that composes segments

// What a block works on: channels c .. c + VEC - 1 of sequence b, rows
// [r0, r1) of segment seg.  Blocks that share cache lines of a row go to the
// same XCD (blocks are dealt to the 8 XCDs in turn).  A lane whose channels
// would pass D repeats the last ones (with the same values).
template <int VEC, int RC>
struct Place {
    int64_t b, c, r0, r1, len;
    int before, seg, cl, tl, w, waves;
    __device__ __forceinline__ Place(const kan_recur_desc_t& d, const RecurPlan& p, const int32_t* lengths) {
        const unsigned n = gridDim.x, i = blockIdx.x;
        unsigned l = n % 8 == 0 ? i % 8 * (n / 8) + i / 8 : i;
        const unsigned cb = l % p.blocks;
        l /= p.blocks;
        seg = (int)(l % p.segs);
        b = l / p.segs;
        const int lane = threadIdx.x & 63;
        cl = lane % RC;
        tl = lane / RC;
        w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        waves = blockDim.x >> 6;
        const LaneChannels own(cb, cl, RC, VEC, d.D);
        c = own.c;
        before = own.before;
        r0 = seg * p.seg_rows;
        r1 = min(r0 + p.seg_rows, d.T);
        len = length_of(lengths, b, d.T);
    }
};

// Runs of N channels, h -> L h + b: U and L of a channel as a gate's u and f.
template <int N>
struct Run {
    float e[N], b[N];
    // INFINITE: of states that may be infinite, which stay so
    template <bool INFINITE = false>
    __device__ __forceinline__ void apply(float (&h)[N]) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float left = Gate{e[i]}.of_state(h[i]);
            h[i] = (INFINITE && __builtin_isinf(h[i]) ? h[i] : left) + b[i];
        }
    }
};

// A tile's runs, wave by wave, and the state at its start.
template <int VEC, int RC>
struct Tile {
    Run<VEC> of[RW][RC];
    float start[RC][VEC];
};

// The same while runs are composed.  A tile's rows add to b by f and L as they
// are rounded: that moves a contribution by some last places once, as the
// state goes on from tile to tile by Run::apply.
template <int N>
struct Rows {
    float U[N], L[N], b[N];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < N; ++i) U[i] = b[i] = 0.0f, L[i] = 1.0f;
    }
    __device__ __forceinline__ void step(int i, Shares q, float x) {
        b[i] = __builtin_fmaf(q.f, b[i], q.u * x);
        then(i, q);
    }
    __device__ __forceinline__ void back(int i, Shares q, float d) {
        b[i] = q.f * (d + b[i]);
        then(i, q);
    }
    // the rows of `before`, then these
    __device__ __forceinline__ void after(const Rows& before) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            b[i] = __builtin_fmaf(L[i], before.b[i], b[i]);
            U[i] = __builtin_fmaf(U[i], before.L[i], before.U[i]);
            L[i] *= before.L[i];
        }
    }
    __device__ __forceinline__ Run<N> run() const {
        Run<N> o;
#pragma unroll
        for (int i = 0; i < N; ++i) o.e[i] = Gate::of(Shares{U[i], L[i]}).e, o.b[i] = b[i];
        return o;
    }

private:
    __device__ __forceinline__ void then(int i, Shares q) {
        U[i] = __builtin_fmaf(q.u, L[i], U[i]);
        L[i] *= q.f;
    }
};

// v of the lane k before this one in the order of the scan
template <bool BACK>
__device__ __forceinline__ float earlier(float v, int k) {
    return BACK ? __shfl_down(v, k, 64) : __shfl_up(v, k, 64);
}

// Composes a wave's lanes, in row order (forward) or against it (BACK): the
// runs up to and with each lane.
template <int VEC, int RC, bool BACK>
__device__ __forceinline__ void scan_wave(Rows<VEC>& rows, const Place<VEC, RC>& at) {
    constexpr int RL = 64 / RC;
    const int place = BACK ? RL - 1 - at.tl : at.tl;
#pragma unroll
    for (int k = 1; k < RL; k *= 2) {
        Rows<VEC> o;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            o.U[i] = earlier<BACK>(rows.U[i], k * RC);
            o.L[i] = earlier<BACK>(rows.L[i], k * RC);
            o.b[i] = earlier<BACK>(rows.b[i], k * RC);
        }
        if (place >= k) rows.after(o);
    }
}

// Scan of the block's runs: h, the state at the tile's start, becomes the state
// at its end, and `mine` the state at the start of the lane's rows.  Where the
// end is not finite it is done again with care for infinities (that care for
// every run: 8 x 4096 x 2048 bf16 forward 104.3 -> 106.3 us, 4 x 1000 x 512 float32
// 17.2 -> 17.8; none at all 102.9 and 16.7).
template <int VEC, int RC, bool BACK>
__device__ __forceinline__ void scan_tile(Rows<VEC> rows, float (&h)[VEC], float (&mine)[VEC],
                                          const Place<VEC, RC>& at, Tile<VEC, RC>& tot) {
    constexpr int RL = 64 / RC;
    scan_wave<VEC, RC, BACK>(rows, at);
    const Run<VEC> run = rows.run();
    if (at.tl == (BACK ? 0 : RL - 1)) {
        tot.of[at.w][at.cl] = run;
        if (at.w == 0)
#pragma unroll
            for (int i = 0; i < VEC; ++i) tot.start[at.cl][i] = h[i];
    }
    Run<VEC> o;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        o.e[i] = earlier<BACK>(run.e[i], RC);
        o.b[i] = earlier<BACK>(run.b[i], RC);
    }
    if (at.tl == (BACK ? RL - 1 : 0)) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) o.e[i] = o.b[i] = 0.0f;
    }
    __syncthreads();
    auto wave = [&](int k, auto infinite) {
        const int q = BACK ? at.waves - 1 - k : k;
#pragma unroll
        for (int i = 0; i < VEC; ++i) mine[i] = k == 0 || q == at.w ? h[i] : mine[i];
        tot.of[q][at.cl].template apply<infinite.value>(h);
    };
    if (at.waves == RW)
#pragma unroll
        for (int k = 0; k < RW; ++k) wave(k, std::false_type());
    else
        for (int k = 0; k < at.waves; ++k) wave(k, std::false_type());
    bool fine = true;
#pragma unroll
    for (int i = 0; i < VEC; ++i) fine = fine && __builtin_isfinite(h[i]);
    if (!__all(fine)) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) h[i] = tot.start[at.cl][i];
#pragma unroll 1
        for (int k = 0; k < at.waves; ++k) wave(k, std::true_type());
    }
    o.template apply<true>(mine);
}

// Element i of a row pointer's vector at row t.
template <typename TS, int VEC>
__device__ __forceinline__ Raw<TS, VEC> row_at(const TS* p, int64_t t, int64_t stride) {
    return load_raw<TS, VEC>(p + t * stride);
}

// h after the runs of the segments before this one (after it, BACK), from the
// launch that composed them: each of the block's runs of lanes composes a
// share of them, and the shares are scanned like a tile's.
template <int VEC, int RC, bool BACK>
__device__ __forceinline__ void from_segments(const RecurPlan& p, const Place<VEC, RC>& at, int64_t D,
                                              const float* runs, float (&h)[VEC],
                                              Tile<VEC, RC>& tot) {
    const int groups = at.waves * (64 / RC), g = at.w * (64 / RC) + at.tl;
    const int n = BACK ? p.segs - 1 - at.seg : at.seg, each = (n + groups - 1) / groups;
    const int k0 = (BACK ? groups - 1 - g : g) * each, k1 = min(k0 + each, n);
    Rows<VEC> rows;
    rows.clear();
    for (int k = k0; k < k1; ++k) {
        const float* r = runs + ((at.b * p.segs + (BACK ? p.segs - 1 - k : k)) * 2) * D + at.c;
        const Raw<float, VEC> e = load_raw<float, VEC>(r), bb = load_raw<float, VEC>(r + D);
        Rows<VEC> one;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const Shares q = Gate{raw_value(e, i)}.shares();
            one.U[i] = q.u, one.L[i] = q.f, one.b[i] = raw_value(bb, i);
        }
        one.after(rows);
        rows = one;
    }
    float mine[VEC];
    scan_tile<VEC, RC, BACK>(rows, h, mine, at, tot);
}

// Rows' loads are waited for here, not where they are used.
template <typename TS, int VEC, int N>
__device__ __forceinline__ void arrived(Raw<TS, VEC> (&rows)[N]) {
#pragma unroll
    for (int r = 0; r < N; ++r)
#pragma unroll
        for (uint32_t& w : rows[r].w) asm volatile("" : "+v"(w));
}
template <int VEC>
__device__ __forceinline__ void load_state(const float* from, int64_t at, float (&h)[VEC]) {
    Raw<float, VEC> r;
    if (from) r = load_raw<float, VEC>(from + at);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        h[i] = from ? raw_value(r, i) : 0.0f;
        // has arrived here: a wait where the tiles' loop uses it would, in every
        // tile, be one for the next tile's loads
        asm volatile("" : "+v"(h[i]));
    }
}

constexpr int RF = kRecurRows, RB = kRecurRows;    // rows of a lane in a tile

// Infinities and NaN among the rows that a segment's run leaves out would end
// with their segment.  A block marks the channels whose last state has one, and
// a third launch (AGAIN) of blocks that return at once where nothing is marked
// goes through the marked channels' sequences whole and stores these alone.  So
// a result does not depend on whether its sequence was cut, for 3 us a call (a
// launch that finds nothing).  marks: [B][D].
template <int VEC>
__device__ __forceinline__ void mark(int* marks, const float (&h)[VEC]) {
#pragma unroll
    for (int i = 0; i < VEC; ++i)
        if (!__builtin_isfinite(h[i])) marks[i] = 1;
}
template <int VEC>
struct Marked {
    bool own[VEC];
    bool none;                    // of the block's channels: the same in all of its waves, which have them all
    __device__ __forceinline__ Marked(const int* marks) {
        bool any = false;
#pragma unroll
        for (int i = 0; i < VEC; ++i) own[i] = marks[i] != 0, any = any || own[i];
        none = !__any(any);
    }
    __device__ __forceinline__ void put(float* p, const float (&v)[VEC]) const {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (own[i]) p[i] = v[i];
    }
    __device__ __forceinline__ void put(uint16_t* p, const float (&v)[VEC]) const {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (own[i]) p[i] = f2bf(v[i]);
    }
};

// The runs of the segments, for the launch that starts each segment from them:
// of h from x and g, or (BACK) of c from dy and g.  A segment's run is composed
// from the end that counts most, the one where it hands its state on, and ends
// where the share that is left of what comes before is at most 2^-64 in every
// channel of the block: less than half a last place of what follows, unless the
// state that is dropped was 2^40 times as large.  (2^-25 is half a last place of
// a state of the same size, and 7 us less; but what is left of one
// large input would then end at a segment's start.)  Common gates forget in a
// tile or two (128 rows by 64 channels); gates that do not are read to the
// segment's start.
template <typename TS, typename TV, int VEC, int RC, bool BACK>
__global__ void __launch_bounds__(64 * RW) recur_runs_kernel(kan_recur_desc_t d, RecurPlan p, const TS* g, const TV* v,
                                                             int64_t v_row, int64_t v_seq, const int32_t* lengths,
                                                             float* runs, int* marks) {
    __shared__ Rows<VEC> tot[2][RW][RC];
    constexpr int RL = 64 / RC;
    const Place<VEC, RC> at(d, p, lengths);
    g += at.b * d.g_seq + at.c;
    v += at.b * v_seq + at.c;
    if (const int64_t i = (int64_t)blockIdx.x * 64 + threadIdx.x; threadIdx.x < 64 && i < d.B * d.D) marks[i] = 0;
    const int tile = at.waves * RL * RF, first = (at.w * RL + at.tl) * RF;
    const int64_t inside = min(at.len, at.r1), tiles = max((int64_t)0, (inside - at.r0 + tile - 1) / tile);
    Raw<TS, VEC> gr[RF];
    Raw<TV, VEC> vr[RF];
    auto load = [&](int64_t t0) {                      // rows past the length repeat its last one
#pragma unroll
        for (int r = 0; r < RF; ++r) {
            const int64_t q = min(t0 + first + r, at.len - 1);
            gr[r] = row_at<TS, VEC>(g, q, d.g_row);
            vr[r] = row_at<TV, VEC>(v, q, v_row);
        }
    };
    auto start = [&](int64_t k) { return at.r0 + (BACK ? k : tiles - 1 - k) * tile; };
    Rows<VEC> all;
    all.clear();
    for (int64_t k = 0; k < tiles; ++k) {
        const int64_t t = start(k) + first;
        load(start(k));
        Rows<VEC> rows;
        rows.clear();
#pragma unroll
        for (int j = 0; j < RF; ++j) {
            const int r = BACK ? RF - 1 - j : j;
            const bool in = t + r < inside;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const Shares q = in ? Shares::of(raw_value(gr[r], i)) : Shares::idle();
                const float x = in ? raw_value(vr[r], i) : 0.0f;
                BACK ? rows.back(i, q, x) : rows.step(i, q, x);
            }
        }
        scan_wave<VEC, RC, BACK>(rows, at);
        if (at.tl == (BACK ? 0 : RL - 1)) tot[k & 1][at.w][at.cl] = rows;
        __syncthreads();
        for (int q = 0; q < at.waves; ++q) all.after(tot[k & 1][BACK ? q : at.waves - 1 - q][at.cl]);
        bool done = true;
#pragma unroll
        for (int i = 0; i < VEC; ++i) done = done && all.L[i] <= 0x1p-64f;
        // a wave has all of the block's channels and the same runs of them as
        // every other wave: they leave together
        if (__all(done)) break;
    }
    if (at.w != 0 || at.tl != 0) return;
    const Run<VEC> run = all.run();
    runs += (at.b * p.segs + at.seg) * 2 * d.D + at.c;
    if (at.before == 0) {
        store_vec<VEC>(runs, run.e);
        store_vec<VEC>(runs + d.D, run.b);
        return;
    }
    // the channel block before this one stores its own, which end where its
    // channels let them and may differ from these in what 2^-64 is worth
#pragma unroll
    for (int i = 0; i < VEC; ++i)
        if (i >= at.before) runs[i] = run.e[i], runs[d.D + i] = run.b[i];
}

// Forward.  Two blocks to a compute unit (at most 128 registers): 32 x 700 x 770
// float32 47.0 -> 45.5 us, 64 x 300 x 768 39.9 -> 38.1, 4 x 1000 x 512 12.1 ->
// 12.8.
template <typename TS, int VEC, int RC, bool STREAM, bool AGAIN>
__global__ void __launch_bounds__(64 * RW, 4) recur_fwd_kernel(kan_recur_desc_t d, RecurPlan p, RecurArgs a,
                                                            const float* runs, int* marks) {
    __shared__ Tile<VEC, RC> tot[2];
    constexpr int RL = 64 / RC;
    const Place<VEC, RC> at(d, p, a.lengths);
    const int64_t D = d.D;
    typename std::conditional<AGAIN, Marked<VEC>, const int*>::type marked(marks + at.b * D + at.c);
    if constexpr (AGAIN)
        if (marked.none) return;
    auto put = [&](float* to, const float (&v)[VEC]) {
        if constexpr (AGAIN) marked.put(to, v);
        else store_vec<VEC, STREAM>(to, v);
    };
    auto put_last = [&](const float (&v)[VEC]) {
        if constexpr (AGAIN) marked.put(a.hT + at.b * D + at.c, v);
        else store_vec<VEC>(a.hT + at.b * D + at.c, v);
    };
    const TS* x = static_cast<const TS*>(a.x) + at.b * d.x_seq + at.c;
    const TS* g = static_cast<const TS*>(a.g) + at.b * d.g_seq + at.c;
    float* y = a.out + at.b * d.T * D + at.c;
    float h[VEC];
    load_state<VEC>(a.h0, at.b * D + at.c, h);
    if (p.segs > 1) from_segments<VEC, RC, false>(p, at, D, runs, h, tot[1]);
    const int tile = at.waves * RL * RF, first = (at.w * RL + at.tl) * RF;
    const int64_t inside = min(at.len, at.r1);
    Raw<TS, VEC> xr[RF], gr[RF];
    auto load = [&](int64_t t0, auto checked) {
#pragma unroll
        for (int r = 0; r < RF; ++r) {
            const int64_t t = t0 + first + r, q = checked.value ? min(t, at.len - 1) : t;
            gr[r] = row_at<TS, VEC>(g, q, d.g_row);
            xr[r] = row_at<TS, VEC>(x, q, d.x_row);
        }
    };
    // h from 0 at the lane's first row; from the state before it, a row's is this
    // and what is left of that state
    Rows<VEC> rows;
    float f[RF][VEC], own[RF][VEC], start[VEC];
    auto compose = [&](int64_t t, auto checked) {
        rows.clear();
#pragma unroll
        for (int r = 0; r < RF; ++r) {
            const bool in = !checked.value || t + r < inside;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const Shares q = in ? Shares::of(raw_value(gr[r], i)) : Shares::idle();
                rows.step(i, q, in ? raw_value(xr[r], i) : 0.0f);
                f[r][i] = q.f;
                own[r][i] = rows.b[i];
            }
        }
    };
    auto row = [&](int r, float (&o)[VEC]) {           // rows in order
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            start[i] *= f[r][i];
            o[i] = start[i] + own[r][i];
        }
    };
    int64_t t0 = at.r0;
    int parity = 0;
    bool ready = t0 + tile <= inside;
    if (ready) {
        load(t0, std::false_type());
        arrived(gr), arrived(xr);
    }
    // The whole tiles that another one follows.  The next one's loads have the
    // time of the scan, the stores that of the next tile up to its scan's end:
    // were the loads waited for after the stores are issued, the wait would be
    // one for the stores too.
    for (; t0 + 2 * tile <= inside; t0 += tile, parity ^= 1) {
        compose(t0 + first, std::false_type());
        __builtin_amdgcn_sched_barrier(0);
        load(t0 + tile, std::false_type());
        scan_tile<VEC, RC, false>(rows, h, start, at, tot[parity]);
        arrived(gr), arrived(xr);
#pragma unroll
        for (int r = 0; r < RF; ++r) {
            float o[VEC];
            row(r, o);
            put(y + (t0 + first + r) * D, o);
        }
    }
    for (; t0 < inside; t0 += tile, parity ^= 1, ready = false) {      // the last ones
        const int64_t t = t0 + first;
        if (!ready) load(t0, std::true_type());
        compose(t, std::true_type());
        scan_tile<VEC, RC, false>(rows, h, start, at, tot[parity]);
#pragma unroll
        for (int r = 0; r < RF; ++r) {
            float o[VEC];
            row(r, o);
            if (a.hT && t + r == at.len - 1) put_last(o);     // the bits of y
#pragma unroll
            for (int i = 0; i < VEC; ++i) o[i] = t + r < at.len ? o[i] : 0.0f;
            if (t + r < at.r1) put(y + (t + r) * D, o);
        }
    }
    for (; t0 < at.r1; t0 += tile) {                   // rows past the length
        const float zero[VEC] = {};
#pragma unroll
        for (int r = 0; r < RF; ++r)
            if (t0 + first + r < at.r1) put(y + (t0 + first + r) * D, zero);
    }
    if (a.hT && at.len == 0 && at.seg == 0 && at.w == 0 && at.tl == 0) put_last(h);     // h0
    if (at.seg + 1 < p.segs && at.w == 0 && at.tl == 0) mark(marks + at.b * D + at.c, h);
}

// Backward: the same, from the last row of a segment to its first, and with two
// blocks to a compute unit (130 registers: 32 x 700 x 770 float32 103 -> 113 us).
template <typename TS, typename TG, int VEC, int RC, bool STREAM, bool AGAIN>
__global__ void __launch_bounds__(64 * RW, 4) recur_bwd_kernel(kan_recur_desc_t d, RecurPlan p, RecurArgs a,
                                                            const float* runs, int* marks) {
    __shared__ Tile<VEC, RC> tot[2];
    constexpr int RL = 64 / RC;
    const Place<VEC, RC> at(d, p, a.lengths);
    const int64_t D = d.D;
    typename std::conditional<AGAIN, Marked<VEC>, const int*>::type marked(marks + at.b * D + at.c);
    if constexpr (AGAIN)
        if (marked.none) return;
    auto put = [&](TG* to, const float (&v)[VEC]) {
        if constexpr (AGAIN) marked.put(to, v);
        else store_vec<VEC, STREAM>(to, v);
    };
    const TS* x = static_cast<const TS*>(a.x) + at.b * d.x_seq + at.c;
    const TS* g = static_cast<const TS*>(a.g) + at.b * d.g_seq + at.c;
    const float* y = a.y + at.b * d.T * D + at.c;
    const float* dy = a.dy + at.b * d.T * D + at.c;
    const bool grads = a.dx;
    TG* dx = grads ? static_cast<TG*>(a.dx) + at.b * d.dx_seq + at.c : nullptr;
    TG* dg = grads ? static_cast<TG*>(a.dg) + at.b * d.dg_seq + at.c : nullptr;
    float c[VEC];
    load_state<VEC>(a.dhT, at.b * D + at.c, c);
    if (p.segs > 1) from_segments<VEC, RC, true>(p, at, D, runs, c, tot[1]);
    const int tile = at.waves * RL * RB, first = (at.w * RL + at.tl) * RB;
    int parity = 0;
    const int64_t tiles = (at.r1 - at.r0 + tile - 1) / tile;
    for (int64_t k = tiles - 1; k >= 0; --k) {
        const int64_t t0 = at.r0 + k * tile, t = t0 + first;
        if (t0 >= at.len) {                            // uniform: rows past the length
            if (!grads) continue;
            const float zero[VEC] = {};
#pragma unroll
            for (int r = 0; r < RB; ++r)
                if (t + r < at.r1) {
                    put(dx + (t + r) * d.dx_row, zero);
                    put(dg + (t + r) * d.dg_row, zero);
                }
            continue;
        }
        Rows<VEC> rows;
        rows.clear();
        Gate e[RB][VEC];
        float dv[RB][VEC], diff[RB][VEC];              // dy; h_{t-1} - x_t
        const bool whole = t0 > 0 && t0 + tile <= min(at.len, at.r1);    // uniform
        auto load = [&](auto checked) {
            Raw<TS, VEC> xr[RB], gr[RB];
            Raw<float, VEC> yr[RB], dr[RB];
#pragma unroll
            for (int r = 0; r < RB; ++r) {
                const int64_t q = checked.value ? min(t + r, at.len - 1) : t + r;
                gr[r] = row_at<TS, VEC>(g, q, d.g_row);
                dr[r] = row_at<float, VEC>(dy, q, D);
                if (grads) {
                    xr[r] = row_at<TS, VEC>(x, q, d.x_row);
                    yr[r] = row_at<float, VEC>(y, checked.value ? max(q - 1, (int64_t)0) : q - 1, D);
                }
            }
#pragma unroll
            for (int r = RB - 1; r >= 0; --r) {
                const bool in = !checked.value || (t + r < at.len && t + r < at.r1);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    e[r][i] = in ? Gate::of(raw_value(gr[r], i)) : Gate::idle();
                    dv[r][i] = in ? raw_value(dr[r], i) : 0.0f;
                    if (grads) {
                        const float before = !checked.value || t + r > 0 ? raw_value(yr[r], i)
                                             : a.h0                      ? a.h0[at.b * D + at.c + i]
                                                                         : 0.0f;
                        diff[r][i] = in ? before - raw_value(xr[r], i) : 0.0f;
                    }
                }
            }
        };
        if (whole) load(std::false_type());
        else load(std::true_type());
#pragma unroll
        for (int r = RB - 1; r >= 0; --r)
#pragma unroll
            for (int i = 0; i < VEC; ++i) rows.back(i, e[r][i].shares(), dv[r][i]);
        float s[VEC];
        scan_tile<VEC, RC, true>(rows, c, s, at, tot[parity]);
        parity ^= 1;
        if (!grads) continue;
#pragma unroll
        for (int r = RB - 1; r >= 0; --r) {
            float ox[VEC], og[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const Shares q = e[r][i].shares();
                const float del = dv[r][i] + s[i];
                ox[i] = q.u * del;
                og[i] = q.f * diff[r][i] * ox[i];
                s[i] = q.f * del;
            }
            if (t + r < at.r1) {
                if (t + r >= at.len)
#pragma unroll
                    for (int i = 0; i < VEC; ++i) ox[i] = og[i] = 0.0f;
                put(dx + (t + r) * d.dx_row, ox);
                put(dg + (t + r) * d.dg_row, og);
            }
        }
    }
    if (a.dh0 && at.seg == 0 && at.w == 0 && at.tl == 0) {
        if constexpr (AGAIN) marked.put(a.dh0 + at.b * D + at.c, c);
        else store_vec<VEC>(a.dh0 + at.b * D + at.c, c);
    }
    if (at.seg > 0 && at.w == 0 && at.tl == 0) mark(marks + at.b * D + at.c, c);
}

// One row of each sequence.  Slots differ, so no two threads share a state
// element; the last vector of a row is cut, not moved back, because state is
// read and written.
template <typename TS>
__global__ void __launch_bounds__(64) recur_step_kernel(kan_recur_desc_t d, int64_t S, const TS* x, const TS* g,
                                                        float* state, const int32_t* slots, float* y) {
    const unsigned cb = (unsigned)((d.D + 63) / 64);
    const int64_t b = blockIdx.x / cb, c = (int64_t)(blockIdx.x % cb) * 64 + threadIdx.x;
    if (c >= d.D) return;
    const int64_t slot = slots ? (int64_t)slots[b] : b;
    if (slot < 0 || slot >= S) {
        y[b * d.D + c] = 0.0f;
        return;
    }
    float* st = state + slot * d.D + c;
    const float n = Gate::of(load_f(g, b * d.g_seq + c)).step(*st, load_f(x, b * d.x_seq + c));
    *st = n;
    y[b * d.D + c] = n;
}

// The plan of the launch that composes the segments' runs: lanes and waves of
// its own, the same segments.
RecurPlan runs_plan(const kan_recur_desc_t& d, RecurPlan p) {
    p.lanes = kRunsLanes(p.vec);
    p.blocks = (unsigned)((d.D + p.lanes * p.vec - 1) / (p.lanes * p.vec));
    p.waves = 1;
    while (p.waves < kRecurWaves && p.waves * kRecurRows * (64 / p.lanes) < p.seg_rows) p.waves *= 2;
    return p;
}

// That of the launch which goes through marked channels: whole sequences.
RecurPlan again_plan(const kan_recur_desc_t& d, RecurPlan p) {
    p.segs = 1;
    p.seg_rows = d.T;
    return runs_plan(d, p);
}

template <typename TS, int VEC, int RC, bool STREAM = false>
hipError_t fwd_t(const kan_recur_desc_t& d, const RecurPlan& p, const RecurArgs& a, char* ws, hipStream_t s) {
    float* runs = reinterpret_cast<float*>(ws);
    int* marks = reinterpret_cast<int*>(ws + p.off_marks);
    const dim3 grid((unsigned)(d.B * p.blocks * p.segs)), block(64 * p.waves);
    if (p.segs > 1) {
        const RecurPlan r = runs_plan(d, p);
        hipLaunchKernelGGL((recur_runs_kernel<TS, TS, VEC, kRunsLanes(VEC), false>),
                           dim3((unsigned)(d.B * r.blocks * r.segs)), dim3(64 * r.waves), 0, s, d, r,
                           static_cast<const TS*>(a.g), static_cast<const TS*>(a.x), d.x_row, d.x_seq, a.lengths,
                           runs, marks);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((recur_fwd_kernel<TS, VEC, RC, STREAM, false>), grid, block, 0, s, d, p, a, runs, marks);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.segs == 1) return e;
    const RecurPlan w = again_plan(d, p);
    hipLaunchKernelGGL((recur_fwd_kernel<TS, VEC, kRunsLanes(VEC), false, true>), dim3((unsigned)(d.B * w.blocks)),
                       dim3(64 * w.waves), 0, s, d, w, a, nullptr, marks);
    return hipGetLastError();
}

template <typename TS, typename TG, int VEC, int RC, bool STREAM = false>
hipError_t bwd_t(const kan_recur_desc_t& d, const RecurPlan& p, const RecurArgs& a, char* ws, hipStream_t s) {
    float* runs = reinterpret_cast<float*>(ws);
    int* marks = reinterpret_cast<int*>(ws + p.off_marks);
    const dim3 grid((unsigned)(d.B * p.blocks * p.segs)), block(64 * p.waves);
    if (p.segs > 1) {
        const RecurPlan r = runs_plan(d, p);
        hipLaunchKernelGGL((recur_runs_kernel<TS, float, VEC, kRunsLanes(VEC), true>),
                           dim3((unsigned)(d.B * r.blocks * r.segs)), dim3(64 * r.waves), 0, s, d, r,
                           static_cast<const TS*>(a.g), a.dy, d.D, d.T * d.D, a.lengths, runs, marks);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((recur_bwd_kernel<TS, TG, VEC, RC, STREAM, false>), grid, block, 0, s, d, p, a, runs, marks);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.segs == 1) return e;
    const RecurPlan w = again_plan(d, p);
    hipLaunchKernelGGL((recur_bwd_kernel<TS, TG, VEC, kRunsLanes(VEC), false, true>), dim3((unsigned)(d.B * w.blocks)),
                       dim3(64 * w.waves), 0, s, d, w, a, nullptr, marks);
    return hipGetLastError();
}

// Large outputs are stored as streamed data where rows start on cache lines (8 x
// 4096 x 2048: bf16 forward 106.5 -> 104 us, float32 backward 327 -> 315.5); cut
// lines make streamed stores slower (70 x 1531 x 770 backward: 529 -> 581).
bool streamed(const kan_recur_desc_t& d, const RecurPlan& p, int64_t bytes) {
    return p.on_lines && d.B * d.T * d.D * bytes >= kStreamBytes;
}

template <typename TS>
hipError_t fwd_v(const kan_recur_desc_t& d, const RecurPlan& p, const RecurArgs& a, char* ws, hipStream_t s) {
    if (p.vec == 1) return fwd_t<TS, 1, 4>(d, p, a, ws, s);
    const bool st = streamed(d, p, 4);
    switch (p.lanes) {
        case 32: return st ? fwd_t<TS, 4, 32, true>(d, p, a, ws, s) : fwd_t<TS, 4, 32>(d, p, a, ws, s);
        case 16: return st ? fwd_t<TS, 4, 16, true>(d, p, a, ws, s) : fwd_t<TS, 4, 16>(d, p, a, ws, s);
        case 8: return fwd_t<TS, 4, 8>(d, p, a, ws, s);
        default: return fwd_t<TS, 4, 4>(d, p, a, ws, s);
    }
}

template <typename TS, typename TG>
hipError_t bwd_v(const kan_recur_desc_t& d, const RecurPlan& p, const RecurArgs& a, char* ws, hipStream_t s) {
    if (p.vec == 1) return bwd_t<TS, TG, 1, 4>(d, p, a, ws, s);
    const bool st = streamed(d, p, sizeof(TG));
    switch (p.lanes) {
        case 32: return st ? bwd_t<TS, TG, 4, 32, true>(d, p, a, ws, s) : bwd_t<TS, TG, 4, 32>(d, p, a, ws, s);
        case 16: return st ? bwd_t<TS, TG, 4, 16, true>(d, p, a, ws, s) : bwd_t<TS, TG, 4, 16>(d, p, a, ws, s);
        case 8: return bwd_t<TS, TG, 4, 8>(d, p, a, ws, s);
        default: return bwd_t<TS, TG, 4, 4>(d, p, a, ws, s);
    }
}

}  // namespace

hipError_t launch_recur_fwd(const kan_recur_desc_t& d, const RecurPlan& p, const RecurArgs& a, char* ws,
                            hipStream_t s) {
    return d.dtype == KAN_F32 ? fwd_v<float>(d, p, a, ws, s) : fwd_v<uint16_t>(d, p, a, ws, s);
}

hipError_t launch_recur_bwd(const kan_recur_desc_t& d, const RecurPlan& p, const RecurArgs& a, char* ws,
                            hipStream_t s) {
    if (d.dtype == KAN_F32)
        return d.grad_dtype == KAN_F32 ? bwd_v<float, float>(d, p, a, ws, s) : bwd_v<float, uint16_t>(d, p, a, ws, s);
    return d.grad_dtype == KAN_F32 ? bwd_v<uint16_t, float>(d, p, a, ws, s)
                                   : bwd_v<uint16_t, uint16_t>(d, p, a, ws, s);
}

hipError_t launch_recur_step(const kan_recur_desc_t& d, int64_t S, const void* x, const void* g, float* state,
                             const int32_t* slots, float* y, hipStream_t s) {
    const dim3 grid((unsigned)((d.D + 63) / 64 * d.B));
    if (d.dtype == KAN_F32)
        hipLaunchKernelGGL(recur_step_kernel<float>, grid, dim3(64), 0, s, d, S,
                           static_cast<const float*>(x), static_cast<const float*>(g), state, slots, y);
    else
        hipLaunchKernelGGL(recur_step_kernel<uint16_t>, grid, dim3(64), 0, s, d, S,
                           static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(g), state, slots, y);
    return hipGetLastError();
}

}  // namespace kan
