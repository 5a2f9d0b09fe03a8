// Embedding lookup with scaling, y[n, :] = s E[id_n, :], and its gradient by
// sorted tokens, dE[v, :] = s sum over n with id_n = v of dy[n, :] (gfx950).
//
// Both move rows and do one operation an element, so HBM traffic bounds them
// (and launches, with few tokens).  The gradient adds no float atomics: a
// first launch lists the rows of every token in ascending order and, in other
// blocks, fills dE with zeros; a second adds the listed rows in chunks - every
// dy row is read once, whatever the tokens' frequencies - and writes the rows
// of the tokens that occur; a third joins tokens that span chunks.  The order
// of every sum depends on the ids alone.  Listing is latency (24 us for 32768
// ids when it runs alone), the fill is bandwidth, so they share a launch; rows
// that occur are written twice, but a fill runs at 6 TB/s where reads and writes
// mixed run at 5.
//
// Measured: lookup of 32768 x 2048 bf16 rows 31 us (5.7 TB/s); gradient of 32768
// x 2048 float32 rows into 65536 185 us (805 MB, 4.4 TB/s: 98 us listing and
// filling, 59 summing at 6 TB/s, 6 joining, the rest between launches).
#include "kan_token.h"
#include "kan_vec.h"

namespace kan {

namespace {

constexpr int EB_T = 256;         // threads of a lookup / summing block
constexpr int ES_W = 16;          // waves of a listing block
constexpr int ES_T = 64 * ES_W;
constexpr int ES_U = 8;           // ids a listing lane loads together
constexpr int EZ_V = 16;          // vectors of zeros that a filling thread writes

// ---- lookup -------------------------------------------------------------------
// Block: 256 / tpr rows at a time, UNR times, tpr lanes of VEC columns to a
// row.  With at least VEC columns the last vector of a row ends at its end
// (it repeats columns of its neighbour, with the same values).
template <typename TE, typename TY, typename TI, int VEC, int UNR, bool STREAM>
__global__ void __launch_bounds__(EB_T) embed_fwd_kernel(const TI* __restrict__ ids, const TE* __restrict__ E,
                                                         TY* __restrict__ y, int64_t N, int64_t V, int64_t D,
                                                         int tpr, float scale) {
    const int lane = threadIdx.x % tpr, sub = threadIdx.x / tpr, rows = EB_T / tpr;
    const int64_t c0 = ((int64_t)blockIdx.y * tpr + lane) * VEC;
    if (c0 >= D) return;
    const int64_t c = c0 + VEC > D ? D - VEC : c0;
    const int64_t n0 = (int64_t)blockIdx.x * rows * UNR + sub;
    int64_t id[UNR];
    Raw<TE, VEC> r[UNR];
#pragma unroll
    for (int q = 0; q < UNR; ++q) {
        const int64_t n = n0 + (int64_t)q * rows;
        id[q] = n < N ? (int64_t)ids[n] : -1;
    }
#pragma unroll
    for (int q = 0; q < UNR; ++q) {
        const bool in = id[q] >= 0 && id[q] < V;
        id[q] = in ? id[q] : -1;
        r[q] = load_raw<TE, VEC>(E + (in ? id[q] : 0) * D + c);
    }
#pragma unroll
    for (int q = 0; q < UNR; ++q) {
        const int64_t n = n0 + (int64_t)q * rows;
        float v[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = id[q] >= 0 ? raw_value(r[q], i) * scale : 0.0f;
        if (n < N) store_vec<VEC, STREAM>(y + n * D + c, v);
    }
}

// ---- listing ------------------------------------------------------------------
// Block r lists the tokens of range r: it reads every id once to count its
// tokens' rows (per wave of the block, each of which takes a contiguous share
// of the ids) and the rows of smaller tokens, which is where its own part of
// the list begins, and a second time to place the rows: place = the token's
// first + rows of it in earlier waves + earlier in this wave.  All sums are of
// integers and every row's place is fixed by the ids.  Each block reads all
// ids, from L2 (N <= 32768: 256 KB): no other block's counts are waited for,
// so one launch is enough.  Its work is N V / 512 ids, whatever D is: 0.9 ms for 2^20
// ids and V = 262144.
//
// The ranges are 16 to a doubling of the token, at most kEmbedWidth wide:
// vocabularies are commonly in the order of frequency, about 1 / rank, and a
// block's time goes with the rows that it places.  With equal ranges the first
// one had half of all rows, and listing 32768 of them took 38 us instead of 24.
__device__ __forceinline__ void range_of(int r, int64_t& lo, int& width) {
    constexpr int N = kEmbedPerDoubling;
    const int doubling = r < N ? 0 : r / N - 1;
    if (doubling < kEmbedDoublings) {
        width = 1 << doubling;
        lo = r < N ? r : (int64_t)(N + r % N) << doubling;
    } else {
        width = kEmbedWidth;
        lo = ((int64_t)N << kEmbedDoublings) + (int64_t)(r - N * (kEmbedDoublings + 1)) * kEmbedWidth;
    }
}

// Blocks past the ranges fill dE, `total` floats, with zeros.
template <typename TI, bool STREAM>
__global__ void __launch_bounds__(ES_T) embed_list_kernel(const TI* __restrict__ ids, int N, int64_t V,
                                                          int2* __restrict__ list, int* __restrict__ start,
                                                          int ranges, float* __restrict__ dE, int64_t total) {
    __shared__ int hist[ES_W][kEmbedWidth];
    __shared__ int sums[ES_W];
    const int t = threadIdx.x, lane = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6);
    if ((int)blockIdx.x >= ranges) {                   // uniform
        const float zero[4] = {};
        int64_t at = ((int64_t)(blockIdx.x - ranges) * (ES_T * EZ_V) + t) * 4;
#pragma unroll
        for (int i = 0; i < EZ_V; ++i, at += ES_T * 4) {
            if (at + 4 <= total) store_vec<4, STREAM>(dE + at, zero);
            else
                for (int64_t k = at; k < total; ++k) dE[k] = 0.0f;
        }
        return;
    }
    int64_t lo;
    int width;
    range_of(blockIdx.x, lo, width);
    const int n_tok = (int)min((int64_t)width, V - lo);
    for (int i = lane; i < n_tok; i += 64) hist[w][i] = 0;
    __syncthreads();
    const int share = ((N + ES_W - 1) / ES_W + 63) / 64 * 64;
    const int a = min((int64_t)w * share, (int64_t)N), b = min((int64_t)a + share, (int64_t)N);
    int below = 0;
    for (int n0 = a; n0 < b; n0 += 64 * ES_U) {
        int64_t id[ES_U];
#pragma unroll
        for (int q = 0; q < ES_U; ++q) {
            const int n = n0 + q * 64 + lane;
            id[q] = n < b ? (int64_t)ids[n] : -1;
        }
#pragma unroll
        for (int q = 0; q < ES_U; ++q) {
            below += id[q] >= 0 && id[q] < lo;
            if (id[q] >= lo && id[q] < lo + n_tok) atomicAdd(&hist[w][(int)(id[q] - lo)], 1);
        }
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) below += __shfl_xor(below, o, 64);
    if (lane == 0) sums[w] = below;
    __syncthreads();
    int first = 0;
#pragma unroll
    for (int i = 0; i < ES_W; ++i) first += sums[i];
    __syncthreads();
    // exclusive scan of the tokens' counts: thread k takes token k
    int count = 0;
    if (t < n_tok)
        for (int i = 0; i < ES_W; ++i) count += hist[i][t];
    int inc = count;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(inc, o, 64);
        if (lane >= o) inc += v;
    }
    if (lane == 63) sums[w] = inc;
    __syncthreads();
    for (int i = 0; i < w; ++i) first += sums[i];
    if (t < n_tok) {
        int at = first + inc - count;
        start[lo + t] = at;
        if (lo + t == V - 1) start[V] = at + count;
        for (int i = 0; i < ES_W; ++i) {
            const int c = hist[i][t];
            hist[i][t] = at;
            at += c;
        }
    }
    __syncthreads();
    for (int n0 = a; n0 < b; n0 += 64 * ES_U) {
        int64_t id[ES_U];
#pragma unroll
        for (int q = 0; q < ES_U; ++q) {
            const int n = n0 + q * 64 + lane;
            id[q] = n < b ? (int64_t)ids[n] : -1;
        }
#pragma unroll
        for (int q = 0; q < ES_U; ++q) {
            const bool in = id[q] >= lo && id[q] < lo + n_tok;
            unsigned long long same = __ballot(in);
            if (same == 0) continue;                   // uniform across the wave
            const int k = in ? (int)(id[q] - lo) : 0;
            // lanes of the same token: those that agree in every bit of k
            uint32_t s0 = (uint32_t)same, s1 = (uint32_t)(same >> 32);
            for (int bit = 0; (1 << bit) < width; ++bit) {
                const int m = (int)((uint32_t)k << (31 - bit)) >> 31;      // the bit, in every place
                const unsigned long long set = __ballot(m != 0);
                s0 &= ~((uint32_t)set ^ (uint32_t)m);
                s1 &= ~((uint32_t)(set >> 32) ^ (uint32_t)m);
            }
            same = ((unsigned long long)s1 << 32) | s0;
            if (in) {
                const int rank = __popcll(same & ((1ull << lane) - 1));
                int* h = &hist[w][k];
                const int at = __hip_atomic_load(h, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP) + rank;
                list[at] = make_int2((int)id[q], n0 + q * 64 + lane);
                // the last lane of the token leaves the next place; a wave's
                // LDS operations are done in order
                if ((same >> lane) == 1)
                    __hip_atomic_store(h, at + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
            }
            __builtin_amdgcn_wave_barrier();
        }
    }
}

// ---- summing ------------------------------------------------------------------
// A chunk of the list: the sum of each token's rows in it.  A token inside the
// chunk is written to dE; one that began in an earlier chunk goes to
// part[chunk][0], one that ends in a later chunk to part[chunk][1].
constexpr int EQ = 8;             // rows loaded together
template <typename TY, int VEC>
__device__ __forceinline__ void sum_chunk(int64_t chunk, int size, int64_t c, const TY* dy, int64_t D,
                                          const int2* list, int total, float scale, float* dE, float* part) {
    if (chunk * size >= total) return;
    const int p0 = (int)chunk * size, p1 = min(p0 + size, total);
    int cur = list[p0].x;                              // {token, row}
    bool head = p0 > 0 && list[p0 - 1].x == cur;
    float acc[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) acc[i] = 0.0f;
    auto put = [&](float* to, float f) {
        float v[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = acc[i] * f, acc[i] = 0.0f;
        store_vec<VEC>(to + c, v);
    };
    float* part0 = part + chunk * 2 * D;
    for (int p = p0; p < p1; p += EQ) {
        int tok[EQ];
        Raw<TY, VEC> r[EQ];
#pragma unroll
        for (int q = 0; q < EQ; ++q) {
            const int at = min(p + q, p1 - 1);
            const int2 e = list[at];
            tok[q] = e.x;
            r[q] = load_raw<TY, VEC>(dy + (int64_t)e.y * D + c);
        }
#pragma unroll
        for (int q = 0; q < EQ; ++q) {
            if (p + q >= p1) break;
            if (tok[q] != cur) {
                head ? put(part0, 1.0f) : put(dE + (int64_t)cur * D, scale);
                head = false;
                cur = tok[q];
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) acc[i] += raw_value(r[q], i);
        }
    }
    const bool tail = p1 < total && list[p1].x == cur;
    if (head) put(part0, 1.0f);
    else if (tail) put(part0 + D, 1.0f);
    else put(dE + (int64_t)cur * D, scale);
}

// 256 / tpr chunks to a block, tpr lanes of VEC columns (blockIdx.y: further columns).
template <typename TY, int VEC>
__global__ void __launch_bounds__(EB_T) embed_sum_kernel(const TY* __restrict__ dy, int64_t V, int64_t D, int tpr,
                                                         int size, const int2* __restrict__ list,
                                                         const int* __restrict__ start, float scale,
                                                         float* __restrict__ dE, float* __restrict__ part) {
    const int lane = threadIdx.x % tpr, sub = threadIdx.x / tpr, rows = EB_T / tpr;
    const int64_t c0 = ((int64_t)blockIdx.y * tpr + lane) * VEC;
    if (c0 >= D) return;
    const int64_t c = c0 + VEC > D ? D - VEC : c0;
    sum_chunk<TY, VEC>((int64_t)blockIdx.x * rows + sub, size, c, dy, D, list, start[V], scale, dE, part);
}

// A token that spans chunks: the sum of its chunks' sums.  Block b looks at
// the boundary of chunks b and b + 1 and joins a token that begins in chunk b
// and goes on.  Four waves add contiguous quarters of the chunks in order,
// then the quarters are added in order.
constexpr int EJ_W = 4;
template <int VEC>
__global__ void __launch_bounds__(64 * EJ_W) embed_join_kernel(int64_t V, int64_t D, int size,
                                                               const int2* __restrict__ list,
                                                               const int* __restrict__ start, float scale,
                                                               float* __restrict__ dE,
                                                               const float* __restrict__ part) {
    __shared__ float quarter[EJ_W][64][VEC];
    const int64_t b = blockIdx.x;
    const int p = (int)((b + 1) * size);
    if (p >= start[V]) return;                         // uniform across the block, as the next one
    const int tok = list[p].x;
    const int first = start[tok], last = (start[tok + 1] - 1) / size;
    if (first >= p || first < p - size) return;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    // pieces: part[b][1], part[b + 1][0], ..., part[last][0]
    const int n = last - (int)b + 1, each = (n + EJ_W - 1) / EJ_W;
    const int q0 = min(w * each, n), q1 = min(q0 + each, n);
    const int64_t c0 = ((int64_t)blockIdx.y * 64 + lane) * VEC;
    const int64_t c = max((int64_t)0, min(c0, D - VEC));
    float acc[VEC] = {};
    for (int q = q0; q < q1; q += EQ) {
        Raw<float, VEC> r[EQ];
#pragma unroll
        for (int k = 0; k < EQ; ++k) {
            const int64_t piece = b + min(q + k, q1 - 1);
            r[k] = load_raw<float, VEC>(part + (piece * 2 + (piece == b)) * D + c);
        }
#pragma unroll
        for (int k = 0; k < EQ; ++k)
            if (q + k < q1)
#pragma unroll
                for (int i = 0; i < VEC; ++i) acc[i] += raw_value(r[k], i);
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) quarter[w][lane][i] = acc[i];
    __syncthreads();
    if (w != 0 || c0 >= D) return;
    float v[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        float s = quarter[0][lane][i];
#pragma unroll
        for (int k = 1; k < EJ_W; ++k) s += quarter[k][lane][i];
        v[i] = s * scale;
    }
    store_vec<VEC>(dE + (int64_t)tok * D + c, v);
}

// lanes of VEC columns to a row: a power of two, at most a block
int lanes_per_row(int64_t D, int vec) {
    int tpr = 1;
    while (tpr < EB_T && (int64_t)tpr * vec < D) tpr *= 2;
    return tpr;
}

template <typename TE, typename TY, typename TI, int VEC>
hipError_t fwd_t(const kan_embed_desc_t& d, const void* ids, const void* E, void* y, hipStream_t s) {
    const int tpr = lanes_per_row(d.D, VEC), rows = EB_T / tpr;
    const unsigned gy = (unsigned)((d.D + (int64_t)tpr * VEC - 1) / ((int64_t)tpr * VEC));
    // four rows to a lane once one row each would fill the GPU's waves several times over
    const bool many = d.N / rows * gy >= 4096;
    const unsigned gx = (unsigned)((d.N + rows * (many ? 4 : 1) - 1) / (rows * (many ? 4 : 1)));
    auto run = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(gx, gy), dim3(EB_T), 0, s, static_cast<const TI*>(ids),
                           static_cast<const TE*>(E), static_cast<TY*>(y), d.N, d.V, d.D, tpr, d.scale);
    };
    // large outputs as streamed data: 32768 x 2048 bf16 36.6 -> 31.3 us
    if (!many) run(embed_fwd_kernel<TE, TY, TI, VEC, 1, false>);
    else if (d.N * d.D * (int64_t)sizeof(TY) < kStreamBytes) run(embed_fwd_kernel<TE, TY, TI, VEC, 4, false>);
    else run(embed_fwd_kernel<TE, TY, TI, VEC, 4, true>);
    return hipGetLastError();
}

template <typename TE, typename TY, int VEC>
hipError_t fwd_i(const kan_embed_desc_t& d, const void* ids, const void* E, void* y, hipStream_t s) {
    if (d.D < VEC)
        return d.id_dtype == KAN_I32 ? fwd_t<TE, TY, int32_t, 1>(d, ids, E, y, s)
                                     : fwd_t<TE, TY, int64_t, 1>(d, ids, E, y, s);
    return d.id_dtype == KAN_I32 ? fwd_t<TE, TY, int32_t, VEC>(d, ids, E, y, s)
                                 : fwd_t<TE, TY, int64_t, VEC>(d, ids, E, y, s);
}

template <typename TY, int VEC>
hipError_t bwd_t(const kan_embed_desc_t& d, const EmbedPlan& p, const void* dy, float* dE, char* ws, hipStream_t s) {
    const int tpr = lanes_per_row(d.D, VEC), rows = EB_T / tpr;
    const unsigned gy = (unsigned)((d.D + (int64_t)tpr * VEC - 1) / ((int64_t)tpr * VEC));
    const int64_t blocks = (p.chunks + rows - 1) / rows;
    int2* list = reinterpret_cast<int2*>(ws + p.off_list);
    int* start = reinterpret_cast<int*>(ws + p.off_start);
    float* part = reinterpret_cast<float*>(ws + p.off_part);
    hipLaunchKernelGGL((embed_sum_kernel<TY, VEC>), dim3((unsigned)blocks, gy), dim3(EB_T), 0, s,
                       static_cast<const TY*>(dy), d.V, d.D, tpr, p.chunk, list, start, d.scale, dE, part);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.chunks == 1) return e;
    const unsigned jy = (unsigned)((d.D + 64 * VEC - 1) / (64 * VEC));
    hipLaunchKernelGGL((embed_join_kernel<VEC>), dim3((unsigned)(p.chunks - 1), jy), dim3(64 * EJ_W), 0, s, d.V, d.D,
                       p.chunk, list, start, d.scale, dE, part);
    return hipGetLastError();
}

template <typename TI, bool STREAM>
hipError_t list_t(const kan_embed_desc_t& d, const EmbedPlan& p, const void* ids, float* dE, char* ws,
                  hipStream_t s) {
    const int64_t total = d.V * d.D, fill = (total + ES_T * EZ_V * 4 - 1) / (ES_T * EZ_V * 4);
    hipLaunchKernelGGL((embed_list_kernel<TI, STREAM>), dim3((unsigned)(p.ranges + fill)), dim3(ES_T), 0, s,
                       static_cast<const TI*>(ids), (int)d.N, d.V,
                       reinterpret_cast<int2*>(ws + p.off_list), reinterpret_cast<int*>(ws + p.off_start),
                       (int)p.ranges, dE, total);
    return hipGetLastError();
}
// A large dE is filled past the caches (537 MB: 207 -> 180 us for the whole
// pass), a small one in them (98 MB: 32 -> 27 us).
template <typename TI>
hipError_t list_s(const kan_embed_desc_t& d, const EmbedPlan& p, const void* ids, float* dE, char* ws,
                  hipStream_t s) {
    return d.V * d.D * 4 >= kStreamBytes ? list_t<TI, true>(d, p, ids, dE, ws, s)
                                         : list_t<TI, false>(d, p, ids, dE, ws, s);
}

}  // namespace

hipError_t launch_embed_fwd(const kan_embed_desc_t& d, const void* ids, const void* E, void* y, hipStream_t s) {
    if (d.dtype == KAN_F32)
        return d.row_dtype == KAN_F32 ? fwd_i<float, float, 4>(d, ids, E, y, s)
                                      : fwd_i<float, uint16_t, 4>(d, ids, E, y, s);
    return d.row_dtype == KAN_F32 ? fwd_i<uint16_t, float, 4>(d, ids, E, y, s)
                                  : fwd_i<uint16_t, uint16_t, 8>(d, ids, E, y, s);
}

hipError_t launch_embed_bwd(const kan_embed_desc_t& d, const EmbedPlan& p, const void* ids, const void* dy, float* dE,
                            char* ws, hipStream_t s) {
    const hipError_t e = d.id_dtype == KAN_I32 ? list_s<int32_t>(d, p, ids, dE, ws, s)
                                                   : list_s<int64_t>(d, p, ids, dE, ws, s);
    if (e != hipSuccess) return e;
    if (d.row_dtype == KAN_F32)
        return d.D < 4 ? bwd_t<float, 1>(d, p, dy, dE, ws, s) : bwd_t<float, 4>(d, p, dy, dE, ws, s);
    return d.D < 4 ? bwd_t<uint16_t, 1>(d, p, dy, dE, ws, s) : bwd_t<uint16_t, 4>(d, p, dy, dE, ws, s);
}

}  // namespace kan
