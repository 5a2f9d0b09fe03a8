// Distillation from a teacher's top logits (gfx950): with p the softmax of a
// row's K teacher logits t / tau and q that of its V student logits z / tau,
//
//     loss = w tau^2 sum_k p_k (log p_k - log q_{id_k})
//     dz_v = dloss w tau (q_v - sum over k with id_k = v of p_k).
//
// K is small beside V: reading z once and writing dz once is the work, so HBM
// traffic bounds it; the arithmetic is an exponential and about six operations
// an element.  A row's maximum m and s = sum exp((z - m) / tau) are kept, not
// their sum in lse: the loss is formed from z_{id} - m and log s, which are
// small where lse and z / tau may be large.
//
// A block takes a row.  In a step it holds the row in registers (up to 16
// vectors of 16 bytes a thread, 256 KB for 1024 threads; what is left of a
// longer row is read again from the caches), so z is read once though its
// gradient needs m and s first; the forward streams the row with a running
// maximum and sum.  The teacher's part is done while the row's loads are in
// flight.
#include "kan_token.h"
#include "kan_vec.h"

namespace kan {

namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int DU = 4;             // vectors that a streaming thread loads together

// Reductions over a block, one barrier each; every call has its own slots.
// Sums go lane by lane and then wave by wave, in a fixed order.
template <int NT>
__device__ __forceinline__ float block_max(float v, float* slots) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
    if (NT == 64) return v;
    if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = v;
    __syncthreads();
    v = slots[0];
#pragma unroll
    for (int i = 1; i < NT / 64; ++i) v = fmaxf(v, slots[i]);
    return v;
}
template <int NT>
__device__ __forceinline__ void block_sum2(float& a, float& b, float* slots) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) a += __shfl_xor(a, o, 64), b += __shfl_xor(b, o, 64);
    if (NT == 64) return;
    if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = a, slots[NT / 64 + (threadIdx.x >> 6)] = b;
    __syncthreads();
    a = slots[0], b = slots[NT / 64];
#pragma unroll
    for (int i = 1; i < NT / 64; ++i) a += slots[i], b += slots[NT / 64 + i];
}

// A row's teacher.  Thread k holds entry k (a block has at least K threads):
// the id (-1: absent or t = -inf), (t - max t) / tau and, after `finish`, p.
template <int NT>
struct Teacher {
    int id;
    float t, p;
    float sum;                    // of exp((t - max) / tau); 0: no entry

    __device__ __forceinline__ void load(const kan_distill_desc_t& d, const DistillArgs& a, int64_t row) {
        id = -1;
        t = -INFINITY;
        if ((int)threadIdx.x >= d.K) return;
        const int64_t at = row * d.K + threadIdx.x;
        const int64_t v = d.id_dtype == KAN_I32 ? (int64_t) static_cast<const int32_t*>(a.ids)[at]
                                                : static_cast<const int64_t*>(a.ids)[at];
        const float x = d.teacher_dtype == KAN_F32 ? static_cast<const float*>(a.t)[at]
                                                   : load_f(static_cast<const uint16_t*>(a.t), at);
        if (v >= 0 && v < d.V && x != -INFINITY) id = (int)v, t = x;
    }
    // ids and p of the row to LDS, p in place
    __device__ __forceinline__ void finish(const kan_distill_desc_t& d, float* slots, int* ids, float* ps) {
        const float m = block_max<NT>(t, slots);       // a NaN shows in the sum
        t = (t - (m == -INFINITY ? 0.0f : m)) / d.tau;
        p = id >= 0 ? exp2f(t * kLog2e) : 0.0f;
        float none = 0.0f;
        sum = p;
        block_sum2<NT>(sum, none, slots + NT / 64);
        p = id >= 0 ? p / sum : 0.0f;
        if ((int)threadIdx.x < d.K) ids[threadIdx.x] = id, ps[threadIdx.x] = p;
        __syncthreads();
    }
    // p becomes the sum over the entries of the same id, at the first of them;
    // the others drop out (id -1)
    __device__ __forceinline__ void join_equal(const kan_distill_desc_t& d, const int* ids, const float* ps) {
        bool first = true;
        float s = 0.0f;
        for (int j = 0; j < d.K; ++j) {
            const bool same = ids[j] == id;
            first = first && !(same && j < (int)threadIdx.x);
            s += same ? ps[j] : 0.0f;
        }
        if (!first) id = -1;
        p = s;
    }
};

// VE elements of a row from element v: -inf past its end.
template <typename TS>
struct Piece {
    static constexpr int VE = 16 / (int)sizeof(TS);
    Raw<TS, VE> r;
    __device__ __forceinline__ void load(const TS* z, int64_t v, int64_t V) {
        if (v + VE <= V) {
            r = load_raw<TS, VE>(z + v);
            return;
        }
        constexpr uint32_t fill = sizeof(TS) == 4 ? 0xff800000u : 0xff80ff80u;
#pragma unroll
        for (int i = 0; i < 4; ++i) r.w[i] = fill;
#pragma unroll
        for (int i = 0; i < VE; ++i) {
            if (v + i >= V) continue;
            if constexpr (sizeof(TS) == 4) r.w[i] = __float_as_uint(z[v + i]);
            else r.w[i / 2] = i & 1 ? (r.w[i / 2] & 0xffffu) | ((uint32_t)z[v + i] << 16)
                                    : (r.w[i / 2] & 0xffff0000u) | z[v + i];
        }
    }
    __device__ __forceinline__ float operator[](int i) const { return raw_value(r, i); }
    __device__ __forceinline__ float max() const {
        float m = (*this)[0];
#pragma unroll
        for (int i = 1; i < VE; ++i) m = fmaxf(m, (*this)[i]);
        return m;
    }
};

__device__ __forceinline__ void put1(float* p, float v) { *p = v; }
__device__ __forceinline__ void put1(uint16_t* p, float v) { *p = f2bf(v); }

template <typename TG, int VE>
__device__ __forceinline__ void put(TG* dz, int64_t v, int64_t V, const float (&o)[VE]) {
    if (v + VE <= V) {
        if constexpr (sizeof(TG) == 4 && VE == 8) {
            const float lo[4] = {o[0], o[1], o[2], o[3]}, hi[4] = {o[4], o[5], o[6], o[7]};
            store_vec<4>(dz + v, lo);
            store_vec<4>(dz + v + 4, hi);
        } else {
            store_vec<VE>(dz + v, o);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < VE; ++i)
        if (v + i < V) put1(dz + v + i, o[i]);
}

// All of a row's (or, from v0 to v1, a part's) gradient zero.
template <typename TG, int NT, int VE>
__device__ __forceinline__ void zeros(TG* dz, int64_t v0, int64_t v1) {
    const float zero[VE] = {};
    for (int64_t v = v0 + threadIdx.x * VE; v < v1; v += NT * VE) put<TG, VE>(dz, v, v1, zero);
}

// Forward (STEP false) and step.  NV vectors of a thread are held in registers.
template <typename TS, typename TG, int NT, int NV, bool STEP>
__global__ void __launch_bounds__(NT) distill_row_kernel(kan_distill_desc_t d, DistillArgs a) {
    constexpr int VE = Piece<TS>::VE, W = NT / 64;
    __shared__ float slots[6 * W];
    __shared__ int ids[kDistillMaxK];
    __shared__ float ps[kDistillMaxK];
    const int64_t row = blockIdx.x, V = d.V;
    const TS* z = static_cast<const TS*>(a.z) + row * d.z_row;
    TG* dz = STEP ? static_cast<TG*>(a.dz) + row * d.dz_row : nullptr;
    const float w = a.w ? a.w[row] : 1.0f;
    if (w == 0.0f) {
        if (threadIdx.x == 0) {
            a.loss[row] = 0.0f;
            if (!STEP) a.lse[row] = 0.0f;
        }
        if (STEP) zeros<TG, NT, VE>(dz, 0, V);
        return;
    }
    const float inv = 1.0f / d.tau, c = kLog2e * inv;
    Teacher<NT> te;
    te.load(d, a, row);
    const int mine = threadIdx.x * VE;
    Piece<TS> keep[NV ? NV : 1];
    float m = -INFINITY, s = 0.0f;
    if (NV) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if ((int64_t)v * NT * VE < V) keep[v].load(z, (int64_t)v * NT * VE + mine, V);    // uniform
    }
    te.finish(d, slots, ids, ps);
    if (STEP) te.join_equal(d, ids, ps);
    // a running maximum and sum over what registers do not hold
    for (int64_t v = (int64_t)NV * NT * VE + mine; v < V; v += (int64_t)NT * VE * DU) {
        Piece<TS> q[DU];
#pragma unroll
        for (int u = 0; u < DU; ++u) q[u].load(z, v + (int64_t)u * NT * VE, V);
        float g = m;
#pragma unroll
        for (int u = 0; u < DU; ++u) g = fmaxf(g, q[u].max());
        const float g0 = g == -INFINITY ? 0.0f : g;
        s *= exp2f((m - g0) * c);
        m = g;
#pragma unroll
        for (int u = 0; u < DU; ++u)
#pragma unroll
            for (int i = 0; i < VE; ++i) s += exp2f((q[u][i] - g0) * c);
    }
    const float m_stream = m;
    if (NV) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if ((int64_t)v * NT * VE < V) m = fmaxf(m, keep[v].max());
    }
    m = block_max<NT>(m, slots + 3 * W);
    const float m0 = m == -INFINITY ? 0.0f : m;
    s *= exp2f((m_stream - m0) * c);
    if (NV) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if ((int64_t)v * NT * VE < V) {
#pragma unroll
                for (int i = 0; i < VE; ++i) {
                    const float e = exp2f((keep[v][i] - m0) * c);
                    s += e;
                    if constexpr (STEP && sizeof(TS) == 4) keep[v].r.w[i] = __float_as_uint(e);
                }
            }
    }
    // sum_k p_k (log p_k + log(teacher's sum) - (z_k - m) / tau); the logs of the sums come after it
    float l = 0.0f, zk = -INFINITY;
    const int k = threadIdx.x;
    if (k < d.K && ids[k] >= 0) {
        zk = load_f(z, ids[k]);
        if (ps[k] != 0.0f) l = ps[k] * (te.t - (zk - m0) * inv);
    }
    block_sum2<NT>(s, l, slots + 4 * W);
    const bool empty = te.sum == 0.0f || s == 0.0f;
    if (threadIdx.x == 0) {
        a.loss[row] = empty ? 0.0f : w * d.tau * d.tau * (l - logf(te.sum) + logf(s));
        if (!STEP) a.lse[row] = m0 * inv + logf(s);
    }
    if (!STEP) return;
    if (empty) {
        zeros<TG, NT, VE>(dz, 0, V);
        return;
    }
    const float f = w * d.tau, fs = f / s;
    if (NV) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if ((int64_t)v * NT * VE < V) {
                float o[VE];
#pragma unroll
                for (int i = 0; i < VE; ++i)
                    o[i] = fs * (sizeof(TS) == 4 ? keep[v][i] : exp2f((keep[v][i] - m0) * c));
                const int64_t at = (int64_t)v * NT * VE + mine;
                if (at < V) put<TG, VE>(dz, at, V, o);
            }
    }
    for (int64_t v = (int64_t)NV * NT * VE + mine; v < V; v += (int64_t)NT * VE * DU) {
        Piece<TS> q[DU];
#pragma unroll
        for (int u = 0; u < DU; ++u) q[u].load(z, v + (int64_t)u * NT * VE, V);
#pragma unroll
        for (int u = 0; u < DU; ++u) {
            float o[VE];
#pragma unroll
            for (int i = 0; i < VE; ++i) o[i] = fs * exp2f((q[u][i] - m0) * c);
            const int64_t at = v + (int64_t)u * NT * VE;
            if (at < V) put<TG, VE>(dz, at, V, o);
        }
    }
    // the teacher's entries again, now with their p taken off
    __syncthreads();
    if (te.id >= 0) put1(dz + te.id, fs * exp2f((zk - m0) * c) - f * te.p);
}

// Backward: block (row, part) writes elements [v0, v1) of a row.
template <typename TS, typename TG, int NT>
__global__ void __launch_bounds__(NT) distill_bwd_kernel(kan_distill_desc_t d, DistillArgs a, int parts,
                                                         int64_t part) {
    constexpr int VE = Piece<TS>::VE, W = NT / 64;
    __shared__ float slots[3 * W];
    __shared__ int ids[kDistillMaxK];
    __shared__ float ps[kDistillMaxK];
    const int64_t row = blockIdx.x / (unsigned)parts, v0 = (blockIdx.x % (unsigned)parts) * part;
    const int64_t v1 = min(v0 + part, d.V);
    const TS* z = static_cast<const TS*>(a.z) + row * d.z_row;
    TG* dz = static_cast<TG*>(a.dz) + row * d.dz_row;
    const float w = a.w ? a.w[row] : 1.0f, lse = w != 0.0f ? a.lse_in[row] : 0.0f;
    if (w == 0.0f || lse == -INFINITY) {
        zeros<TG, NT, VE>(dz, v0, v1);
        return;
    }
    Teacher<NT> te;
    te.load(d, a, row);
    te.finish(d, slots, ids, ps);
    if (te.sum == 0.0f) {
        zeros<TG, NT, VE>(dz, v0, v1);
        return;
    }
    te.join_equal(d, ids, ps);
    const float f = w * d.tau * a.dloss[row], inv = 1.0f / d.tau;
    auto q = [&](float x) { return exp2f(__builtin_fmaf(x, inv, -lse) * kLog2e); };
    for (int64_t v = v0 + threadIdx.x * VE; v < v1; v += (int64_t)NT * VE * DU) {
        Piece<TS> x[DU];
#pragma unroll
        for (int u = 0; u < DU; ++u) x[u].load(z, v + (int64_t)u * NT * VE, v1);
#pragma unroll
        for (int u = 0; u < DU; ++u) {
            float o[VE];
#pragma unroll
            for (int i = 0; i < VE; ++i) o[i] = f * q(x[u][i]);
            const int64_t at = v + (int64_t)u * NT * VE;
            if (at < v1) put<TG, VE>(dz, at, v1, o);
        }
    }
    __syncthreads();
    if (te.id >= v0 && te.id < v1) put1(dz + te.id, f * (q(load_f(z, te.id)) - te.p));
}

template <typename TS, typename TG, int NT, int NV, bool STEP>
hipError_t row_t(const kan_distill_desc_t& d, const DistillArgs& a, hipStream_t s) {
    hipLaunchKernelGGL((distill_row_kernel<TS, TG, NT, NV, STEP>), dim3((unsigned)d.N), dim3(NT), 0, s, d, a);
    return hipGetLastError();
}

// The fewest threads whose registers hold a row, and at least one for each of
// the teacher's entries.
template <typename TS, typename TG>
hipError_t step_t(const kan_distill_desc_t& d, const DistillArgs& a, hipStream_t s) {
    const int64_t per = 16 * Piece<TS>::VE;            // elements that a thread holds
    const int64_t threads = std::max((d.V + per - 1) / per, d.K);
    if (threads <= 64) return row_t<TS, TG, 64, 16, true>(d, a, s);
    if (threads <= 256) return row_t<TS, TG, 256, 16, true>(d, a, s);
    if (threads <= 512) return row_t<TS, TG, 512, 16, true>(d, a, s);
    return row_t<TS, TG, 1024, 16, true>(d, a, s);
}

template <typename TS>
hipError_t fwd_t(const kan_distill_desc_t& d, const DistillArgs& a, hipStream_t s) {
    if (d.K > 256) return row_t<TS, float, 1024, 0, false>(d, a, s);
    if (d.K > 64 || d.V > 64 * 16 * Piece<TS>::VE) return row_t<TS, float, 256, 0, false>(d, a, s);
    return row_t<TS, float, 64, 0, false>(d, a, s);
}

template <typename TS, typename TG, int NT>
hipError_t bwd_n(const kan_distill_desc_t& d, const DistillArgs& a, hipStream_t s) {
    constexpr int VE = Piece<TS>::VE;
    // a few thousand blocks, of at least one round of loads each
    const int64_t parts = std::max<int64_t>(1, std::min<int64_t>((2048 + d.N - 1) / d.N, d.V / (NT * VE * DU)));
    const int64_t part = round_up((d.V + parts - 1) / parts, NT * VE), n = (d.V + part - 1) / part;
    hipLaunchKernelGGL((distill_bwd_kernel<TS, TG, NT>), dim3((unsigned)(d.N * n)), dim3(NT), 0, s, d, a, (int)n,
                       part);
    return hipGetLastError();
}
template <typename TS, typename TG>
hipError_t bwd_t(const kan_distill_desc_t& d, const DistillArgs& a, hipStream_t s) {
    return d.K > 256 ? bwd_n<TS, TG, 1024>(d, a, s) : bwd_n<TS, TG, 256>(d, a, s);
}

}  // namespace

hipError_t launch_distill(const kan_distill_desc_t& d, const DistillPlan&, const DistillArgs& a, char*,
                          hipStream_t s) {
    if (!a.dz) return d.dtype == KAN_F32 ? fwd_t<float>(d, a, s) : fwd_t<uint16_t>(d, a, s);
    if (d.dtype == KAN_F32)
        return d.grad_dtype == KAN_F32 ? step_t<float, float>(d, a, s) : step_t<float, uint16_t>(d, a, s);
    return d.grad_dtype == KAN_F32 ? step_t<uint16_t, float>(d, a, s) : step_t<uint16_t, uint16_t>(d, a, s);
}

hipError_t launch_distill_bwd(const kan_distill_desc_t& d, const DistillArgs& a, hipStream_t s) {
    if (d.dtype == KAN_F32)
        return d.grad_dtype == KAN_F32 ? bwd_t<float, float>(d, a, s) : bwd_t<float, uint16_t>(d, a, s);
    return d.grad_dtype == KAN_F32 ? bwd_t<uint16_t, float>(d, a, s) : bwd_t<uint16_t, uint16_t>(d, a, s);
}

}  // namespace kan
