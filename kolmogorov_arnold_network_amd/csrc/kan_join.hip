// Join between two blocks of a model (gfx950), row by row:
//
//     t = h n1,  n1 = 1 / sqrt(mean(h^2) + eps);   y = r + scale act(gate) w_post t
//     x = w_pre y n2,  n2 = 1 / sqrt(mean(y^2) + eps)
//
// and backward
//
//     z = y n2,  c = w_pre dx,  d = dy + n2 (c - z mean(c z)) = dr
//     e = scale act(gate) d,  dgate = scale act'(gate) w_post t d
//     dh = n1 (w_post e - t mean(w_post e t)),  dw_post = sum e t,  dw_pre = sum dx z.
//
// Each array is read and written once: HBM traffic bounds it.  A row is held in
// the registers of 32 to 1024 threads between its two norms (32768 x 2048 with a
// float32 residual, bf16 else: 144 us, 5.6 TB/s).  In the backward
// pass a block goes through rows of its own and keeps its sums for the weights in
// registers; a second launch adds the blocks' sums in order (32768 x 2048 float32:
// 426 us, 5.0 TB/s).
#include "kan_delta.h"
#include "kan_vec.h"

namespace kan {

namespace {

constexpr int VE = 4;                // elements of a vector

// A thread's vectors of a row: elements VE (lane + L v) .., zero past the end.
template <typename TS, int NVEC, int L>
__device__ __forceinline__ void load_row(const TS* p, int lane, int D, float (&v)[NVEC][VE]) {
#pragma unroll
    for (int i = 0; i < NVEC; ++i) {
        const int at = VE * (lane + L * i);
        if (at + VE <= D) {
            const Raw<TS, VE> r = load_raw<TS, VE>(p + at);
#pragma unroll
            for (int j = 0; j < VE; ++j) v[i][j] = raw_value(r, j);
        } else {
#pragma unroll
            for (int j = 0; j < VE; ++j) v[i][j] = at + j < D ? load_f(p, at + j) : 0.0f;
        }
    }
}
__device__ __forceinline__ void put1(float* p, float v) { *p = v; }
__device__ __forceinline__ void put1(uint16_t* p, float v) { *p = f2bf(v); }
template <typename TS, int NVEC, int L>
__device__ __forceinline__ void store_row(TS* p, int lane, int D, const float (&v)[NVEC][VE]) {
#pragma unroll
    for (int i = 0; i < NVEC; ++i) {
        const int at = VE * (lane + L * i);
        if (at + VE <= D) {
            store_vec<VE>(p + at, v[i]);
        } else {
#pragma unroll
            for (int j = 0; j < VE; ++j)
                if (at + j < D) put1(p + at + j, v[i][j]);
        }
    }
}

// Sum over the L threads of a row, in a fixed order; `slots`: of this call alone.
template <int L>
__device__ __forceinline__ float row_sum(float v, float* slots) {
#pragma unroll
    for (int o = (L < 64 ? L : 64) / 2; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
    if (L <= 64) return v;
    if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = v;
    __syncthreads();
    const int first = threadIdx.x / L * (L / 64);
    v = slots[first];
#pragma unroll
    for (int i = 1; i < L / 64; ++i) v += slots[first + i];
    return v;
}

// act(g) and act'(g), from the smaller of the two shares.  exp(-|g|) is v_exp_f32's 2^t (2^-23)
// of the rounded product t = |g| log2(e), times 1 + ln(2) of what the rounding lost: without that
// factor its error is |g| 2^-24.  From 128 on the smaller share is 0.  The reciprocal is within 2^-23.
// With expf and a division a narrow row's arithmetic takes longer than its bytes (524288 x 128 bf16
// forward 121 us, 102 so).
__device__ __forceinline__ void activation(int kind, float g, float& a, float& slope) {
    const float x = fabsf(g) > 128.0f ? 128.0f : fabsf(g);                     // a NaN stays
    const float t = x * -0x1.715476p0f;
    const float lost = __builtin_fmaf(x, -0x1.4ae0cp-26f, __builtin_fmaf(x, -0x1.715476p0f, -t));
    float e = __builtin_amdgcn_exp2f(t);
    e = __builtin_fmaf(e * lost, 0.693147182f, e);
    const float big = __builtin_amdgcn_rcpf(1.0f + e), small = e * big;
    const float s = g >= 0.0f ? big : small, o = g >= 0.0f ? small : big;      // a NaN is in both
    a = kind == KAN_GATE_SIGMOID ? s : g * s;
    slope = kind == KAN_GATE_SIGMOID ? s * o : s + g * s * o;
}
// 1 / sqrt(sum / D + eps): v_rsq_f32 (2^-23) where its argument is no subnormal number.
__device__ __forceinline__ float factor(float sum, float per, float eps) {
    const float v = __builtin_fmaf(sum, per, eps);
    return v >= 0x1p-120f ? __builtin_amdgcn_rsqf(v) : 1.0f / sqrtf(v);
}

// U rows at a time of each thread's: narrow rows give a wave little to wait for, and a
// block as much work to start as to do (524288 x 128 bf16 with a gate: 119 us with
// one row, 102 with four).
template <typename TH, typename TR, typename TX, int L, int NVEC, int NT, int U>
__global__ void __launch_bounds__(NT) join_fwd_kernel(kan_join_desc_t d, JoinArgs a) {
    __shared__ float slots[2][NT / 64];
    const int lane = threadIdx.x % L, D = (int)d.D;
    const float per = 1.0f / (float)D;
    const int64_t first = (int64_t)blockIdx.x * U * (NT / L) + threadIdx.x / L;
    if (L <= 64 && first >= d.N) return;               // L > 64: a row to a block
    float h[U][NVEC][VE], w[NVEC][VE], y[U][NVEC][VE], g[U][NVEC][VE], n1[U], s[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        int64_t row = first + u * (NT / L);
        if (U > 1 && row >= d.N) row = first;          // read again and not stored
        load_row<TH, NVEC, L>(static_cast<const TH*>(a.h) + row * d.h_row, lane, D, h[u]);
        if (a.gate) load_row<TH, NVEC, L>(static_cast<const TH*>(a.gate) + row * d.gate_row, lane, D, g[u]);
        if (a.r) load_row<TR, NVEC, L>(static_cast<const TR*>(a.r) + row * d.r_row, lane, D, y[u]);
    }
    if (a.w_post) load_row<float, NVEC, L>(a.w_post, lane, D, w);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        n1[u] = 1.0f;
        if (d.flags & KAN_JOIN_POST) {
            float q = 0.0f;
#pragma unroll
            for (int i = 0; i < NVEC; ++i)
#pragma unroll
                for (int j = 0; j < VE; ++j) q = __builtin_fmaf(h[u][i][j], h[u][i][j], q);
            n1[u] = factor(row_sum<L>(q, slots[0]), per, d.eps);
        }
        s[u] = 0.0f;
#pragma unroll
        for (int i = 0; i < NVEC; ++i)
#pragma unroll
            for (int j = 0; j < VE; ++j) {
                float p = h[u][i][j] * n1[u];
                if (a.w_post) p *= w[i][j];
                if (a.gate) {
                    float act, slope;
                    activation(d.activation, g[u][i][j], act, slope);
                    p *= act;
                }
                y[u][i][j] = a.r ? __builtin_fmaf(d.scale, p, y[u][i][j]) : d.scale * p;
                s[u] = __builtin_fmaf(y[u][i][j], y[u][i][j], s[u]);
            }
        const int64_t row = first + u * (NT / L);
        if (U == 1 || row < d.N) store_row<TR, NVEC, L>(static_cast<TR*>(a.y) + row * d.D, lane, D, y[u]);
    }
    if ((d.flags & KAN_JOIN_PRE) && a.w_pre) load_row<float, NVEC, L>(a.w_pre, lane, D, w);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t row = first + u * (NT / L);
        float n2 = 1.0f;
        if (d.flags & KAN_JOIN_PRE) {
            n2 = factor(row_sum<L>(s[u], slots[1]), per, d.eps);
#pragma unroll
            for (int i = 0; i < NVEC; ++i)
#pragma unroll
                for (int j = 0; j < VE; ++j) y[u][i][j] *= a.w_pre ? n2 * w[i][j] : n2;
            if (U == 1 || row < d.N) store_row<TX, NVEC, L>(static_cast<TX*>(a.x) + row * d.D, lane, D, y[u]);
        }
        if (lane == 0 && (U == 1 || row < d.N)) a.stats[row] = n1[u], a.stats[d.N + row] = n2;
    }
}

// Block k has rows k R, k R + 1, .. of every `gridDim.x` R, R = NT / L rows at a time.
template <typename TH, typename TR, typename TX, int L, int NVEC, int NT>
__global__ void __launch_bounds__(NT) join_bwd_kernel(kan_join_desc_t d, JoinArgs a, float* part) {
    __shared__ float slots[4][NT / 64];
    constexpr int R = NT / L;
    const int lane = threadIdx.x % L, D = (int)d.D;
    const float per = 1.0f / (float)D;
    float wq[NVEC][VE], wp[NVEC][VE], sum_post[NVEC][VE], sum_pre[NVEC][VE];
    if (a.w_post) load_row<float, NVEC, L>(a.w_post, lane, D, wq);
    if (a.w_pre) load_row<float, NVEC, L>(a.w_pre, lane, D, wp);
#pragma unroll
    for (int i = 0; i < NVEC; ++i)
#pragma unroll
        for (int j = 0; j < VE; ++j) sum_post[i][j] = sum_pre[i][j] = 0.0f;
    int odd = 0;                                       // slots of one row are free two barriers later
    for (int64_t row = (int64_t)blockIdx.x * R + threadIdx.x / L; row < d.N; row += (int64_t)gridDim.x * R, odd ^= 2) {
        float h[NVEC][VE], y[NVEC][VE], x[NVEC][VE], g[NVEC][VE], e[NVEC][VE];
        load_row<TH, NVEC, L>(static_cast<const TH*>(a.h) + row * d.h_row, lane, D, h);
        if (a.dx) {
            load_row<TR, NVEC, L>(static_cast<const TR*>(a.y_in) + row * d.D, lane, D, y);
            load_row<TX, NVEC, L>(static_cast<const TX*>(a.dx) + row * d.D, lane, D, x);
        }
        if (a.gate) load_row<TH, NVEC, L>(static_cast<const TH*>(a.gate) + row * d.gate_row, lane, D, g);
        if (a.dy) {
            load_row<TR, NVEC, L>(static_cast<const TR*>(a.dy) + row * d.D, lane, D, e);
        } else {
#pragma unroll
            for (int i = 0; i < NVEC; ++i)
#pragma unroll
                for (int j = 0; j < VE; ++j) e[i][j] = 0.0f;
        }
        const float n1 = a.stats_in[row], n2 = a.stats_in[d.N + row];
        if (a.dx) {
            float cz = 0.0f;
#pragma unroll
            for (int i = 0; i < NVEC; ++i)
#pragma unroll
                for (int j = 0; j < VE; ++j) {
                    y[i][j] *= n2;                     // z
                    sum_pre[i][j] = __builtin_fmaf(x[i][j], y[i][j], sum_pre[i][j]);
                    if (a.w_pre) x[i][j] *= wp[i][j];  // c
                    cz = __builtin_fmaf(x[i][j], y[i][j], cz);
                }
            cz = row_sum<L>(cz, slots[odd]) * per;
#pragma unroll
            for (int i = 0; i < NVEC; ++i)
#pragma unroll
                for (int j = 0; j < VE; ++j) e[i][j] = __builtin_fmaf(n2, x[i][j] - y[i][j] * cz, e[i][j]);
        }
        if (a.dr) store_row<TR, NVEC, L>(static_cast<TR*>(a.dr) + row * d.D, lane, D, e);
        float et = 0.0f;
#pragma unroll
        for (int i = 0; i < NVEC; ++i)
#pragma unroll
            for (int j = 0; j < VE; ++j) {
                const float w = a.w_post ? wq[i][j] : 1.0f;
                h[i][j] *= n1;                         // t
                e[i][j] *= d.scale;
                if (a.gate) {
                    float act, slope;
                    activation(d.activation, g[i][j], act, slope);
                    g[i][j] = e[i][j] * w * h[i][j] * slope;
                    e[i][j] *= act;
                }
                sum_post[i][j] = __builtin_fmaf(e[i][j], h[i][j], sum_post[i][j]);
                e[i][j] *= w;
                et = __builtin_fmaf(e[i][j], h[i][j], et);
            }
        if (a.gate && a.dgate) store_row<TH, NVEC, L>(static_cast<TH*>(a.dgate) + row * d.D, lane, D, g);
        if (d.flags & KAN_JOIN_POST) {
            et = row_sum<L>(et, slots[odd + 1]) * per;
#pragma unroll
            for (int i = 0; i < NVEC; ++i)
#pragma unroll
                for (int j = 0; j < VE; ++j) e[i][j] = n1 * (e[i][j] - h[i][j] * et);
        }
        store_row<TH, NVEC, L>(static_cast<TH*>(a.dh) + row * d.D, lane, D, e);
    }
    if (!part) return;
    // the R rows' sums, in order
    __shared__ float sums[R > 1 ? NVEC * VE * L : 1];
    float* out = part + (int64_t)blockIdx.x * 2 * D;
#pragma unroll
    for (int z = 0; z < 2; ++z) {
        float (&mine)[NVEC][VE] = z ? sum_pre : sum_post;
        if (R > 1) {
            for (int k = 1; k < R; ++k) {
                __syncthreads();
                if ((int)threadIdx.x / L == k)
#pragma unroll
                    for (int i = 0; i < NVEC; ++i)
#pragma unroll
                        for (int j = 0; j < VE; ++j) sums[(i * VE + j) * L + lane] = mine[i][j];
                __syncthreads();
                if ((int)threadIdx.x / L == 0)
#pragma unroll
                    for (int i = 0; i < NVEC; ++i)
#pragma unroll
                        for (int j = 0; j < VE; ++j) mine[i][j] += sums[(i * VE + j) * L + lane];
            }
        }
        if ((int)threadIdx.x / L == 0) store_row<float, NVEC, L>(out + z * D, lane, D, mine);
    }
}

// Sums of the blocks' sums: 64 columns to a block, 16 blocks' worth at a time and
// eight such loads on their way (one after the other: 24 us for 1024 blocks of
// 2048 columns, 9 so).
__global__ void __launch_bounds__(1024) join_sum_kernel(const float* part, int64_t D, int blocks, float* dw_post,
                                                        float* dw_pre) {
    __shared__ float sums[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t at = (int64_t)blockIdx.x * 64 + lane;        // of both sums, one after the other
    float v = 0.0f;
    if (at < 2 * D)
        for (int k = wave; k < blocks; k += 16 * 8) {
            float t[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) t[i] = k + 16 * i < blocks ? part[(int64_t)(k + 16 * i) * 2 * D + at] : 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) v += t[i];
        }
    sums[wave][lane] = v;
    __syncthreads();
    if (wave != 0 || at >= 2 * D) return;
    v = sums[0][lane];
#pragma unroll
    for (int k = 1; k < 16; ++k) v += sums[k][lane];
    if (at < D) {
        if (dw_post) dw_post[at] = v;
    } else if (dw_pre) {
        dw_pre[at - D] = v;
    }
}

template <typename TH, typename TR, typename TX, int L, int NVEC, int NT>
hipError_t fwd(const kan_join_desc_t& d, const JoinPlan& p, const JoinArgs& a, hipStream_t s) {
    constexpr int U = NVEC == 1 ? kJoinRows : 1;
    if (U > 1 && p.rows > 1)
        hipLaunchKernelGGL((join_fwd_kernel<TH, TR, TX, L, NVEC, NT, U>), dim3(p.blocks), dim3(NT), 0, s, d, a);
    else
        hipLaunchKernelGGL((join_fwd_kernel<TH, TR, TX, L, NVEC, NT, 1>), dim3(p.blocks), dim3(NT), 0, s, d, a);
    return hipGetLastError();
}
template <typename TH, typename TR, typename TX, int L, int NVEC, int NT>
hipError_t bwd(const kan_join_desc_t& d, const JoinPlan& p, const JoinArgs& a, float* part, hipStream_t s) {
    hipLaunchKernelGGL((join_bwd_kernel<TH, TR, TX, L, NVEC, NT>), dim3(p.blocks), dim3(NT), 0, s, d, a, part);
    return hipGetLastError();
}

// The plan's threads to a row and vectors to a thread, as template arguments.
template <typename TH, typename TR, typename TX>
hipError_t fwd_t(const kan_join_desc_t& d, const JoinPlan& p, const JoinArgs& a, hipStream_t s) {
    switch (p.lanes * 8 + p.vecs) {
        case 32 * 8 + 1: return fwd<TH, TR, TX, 32, 1, 256>(d, p, a, s);
        case 64 * 8 + 1: return fwd<TH, TR, TX, 64, 1, 256>(d, p, a, s);
        case 64 * 8 + 2: return fwd<TH, TR, TX, 64, 2, 256>(d, p, a, s);
        case 64 * 8 + 4: return fwd<TH, TR, TX, 64, 4, 256>(d, p, a, s);
        case 256 * 8 + 2: return fwd<TH, TR, TX, 256, 2, 256>(d, p, a, s);
        case 256 * 8 + 4: return fwd<TH, TR, TX, 256, 4, 256>(d, p, a, s);
        default: return fwd<TH, TR, TX, 1024, 2, 1024>(d, p, a, s);
    }
}
template <typename TH, typename TR, typename TX>
hipError_t bwd_t(const kan_join_desc_t& d, const JoinPlan& p, const JoinArgs& a, float* part, hipStream_t s) {
    switch (p.lanes * 8 + p.vecs) {
        case 32 * 8 + 1: return bwd<TH, TR, TX, 32, 1, 256>(d, p, a, part, s);
        case 64 * 8 + 1: return bwd<TH, TR, TX, 64, 1, 256>(d, p, a, part, s);
        case 64 * 8 + 2: return bwd<TH, TR, TX, 64, 2, 256>(d, p, a, part, s);
        case 256 * 8 + 1: return bwd<TH, TR, TX, 256, 1, 256>(d, p, a, part, s);
        case 256 * 8 + 2: return bwd<TH, TR, TX, 256, 2, 256>(d, p, a, part, s);
        case 256 * 8 + 4: return bwd<TH, TR, TX, 256, 4, 256>(d, p, a, part, s);
        default: return bwd<TH, TR, TX, 1024, 2, 1024>(d, p, a, part, s);
    }
}
template <typename TH, typename TR>
hipError_t fwd_r(const kan_join_desc_t& d, const JoinPlan& p, const JoinArgs& a, hipStream_t s) {
    return d.row_dtype == KAN_F32 ? fwd_t<TH, TR, float>(d, p, a, s) : fwd_t<TH, TR, uint16_t>(d, p, a, s);
}
template <typename TH, typename TR>
hipError_t bwd_r(const kan_join_desc_t& d, const JoinPlan& p, const JoinArgs& a, float* part, hipStream_t s) {
    return d.row_dtype == KAN_F32 ? bwd_t<TH, TR, float>(d, p, a, part, s) : bwd_t<TH, TR, uint16_t>(d, p, a, part, s);
}

}  // namespace

hipError_t launch_join_fwd(const kan_join_desc_t& d, const JoinPlan& p, const JoinArgs& a, hipStream_t s) {
    if (d.dtype == KAN_F32)
        return d.res_dtype == KAN_F32 ? fwd_r<float, float>(d, p, a, s) : fwd_r<float, uint16_t>(d, p, a, s);
    return d.res_dtype == KAN_F32 ? fwd_r<uint16_t, float>(d, p, a, s) : fwd_r<uint16_t, uint16_t>(d, p, a, s);
}

hipError_t launch_join_bwd(const kan_join_desc_t& d, const JoinPlan& p, const JoinArgs& a, char* ws, hipStream_t s) {
    float* part = a.dw_post || a.dw_pre ? reinterpret_cast<float*>(ws) : nullptr;
    hipError_t e = d.dtype == KAN_F32
                       ? (d.res_dtype == KAN_F32 ? bwd_r<float, float>(d, p, a, part, s)
                                                 : bwd_r<float, uint16_t>(d, p, a, part, s))
                       : (d.res_dtype == KAN_F32 ? bwd_r<uint16_t, float>(d, p, a, part, s)
                                                 : bwd_r<uint16_t, uint16_t>(d, p, a, part, s));
    if (e != hipSuccess || !part) return e;
    hipLaunchKernelGGL(join_sum_kernel, dim3((unsigned)((2 * d.D + 63) / 64)), dim3(1024), 0, s, part, d.D,
                       (int)p.blocks, a.dw_post, a.dw_pre);
    return hipGetLastError();
}

}  // namespace kan
