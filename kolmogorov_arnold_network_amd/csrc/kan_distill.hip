// Distillation from a teacher's top logits (gfx950): with p the softmax of a
// row's K teacher logits t / tau and q that of its V student logits z / tau,
//
//     loss = w tau^2 sum_k p_k (log p_k - log q_{id_k})
//     dz_v = dloss w tau (q_v - sum over k with id_k = v of p_k).
//
// K is small beside V: reading z once and writing dz once is the work, one
// or two exponentials an element beside it.  A row's maximum and sum are kept
// relative to each other, s = sum exp((z - m) / tau), and the loss is formed
// from z_{id} - m and log s, which are small where lse and z / tau may be large.
#include "kan_token.h"
#include "kan_vec.h"

namespace kan {

namespace {

constexpr int DT = 256;
constexpr int DW = DT / 64;
constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ float block_max(float v, float* sh) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
    __syncthreads();
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
    __syncthreads();
    v = sh[0];
    for (int i = 1; i < DW; ++i) v = fmaxf(v, sh[i]);
    return v;
}
__device__ __forceinline__ float block_sum(float v, float* sh) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
    __syncthreads();
    v = sh[0];
    for (int i = 1; i < DW; ++i) v += sh[i];
    return v;
}

// The teacher's distribution of a row: ids (-1: absent) and p in LDS; returns
// the maximum of t and the sum of exp((t - max) / tau); the sum is 0 where
// there is no entry.
template <typename TT, typename TI>
__device__ __forceinline__ void teacher(const kan_distill_desc_t& d, const TI* ids, const TT* t, int64_t row, int* id,
                                        float* p, float* sh, float& tm, float& ts) {
    const int K = (int)d.K;
    float m = -INFINITY;
    for (int k = threadIdx.x; k < K; k += DT) {
        const int64_t v = ids[row * K + k];
        const bool in = v >= 0 && v < d.V;
        id[k] = in ? (int)v : -1;
        const float a = in ? load_f(t, row * K + k) : -INFINITY;
        p[k] = a;
        m = fmaxf(m, a);                               // a NaN shows in the sum
    }
    tm = block_max(m, sh);
    float s = 0.0f;
    for (int k = threadIdx.x; k < K; k += DT)
        if (id[k] >= 0 && p[k] != -INFINITY) s += exp2f((p[k] - tm) * (kLog2e / d.tau));
    ts = block_sum(s, sh);
}

template <typename TS, typename TG, typename TT, typename TI, int MODE>      // 0 forward, 1 backward, 2 step
__global__ void __launch_bounds__(DT) distill_kernel(kan_distill_desc_t d, DistillArgs a) {
    __shared__ float sh[DW];
    __shared__ int id[kDistillMaxK];
    __shared__ float p[kDistillMaxK];
    const int64_t row = blockIdx.x;
    const TS* z = static_cast<const TS*>(a.z) + row * d.z_row;
    TG* dz = MODE ? static_cast<TG*>(a.dz) + row * d.dz_row : nullptr;
    const float w = a.w ? a.w[row] : 1.0f;
    float tm = 0.0f, ts = 0.0f, m = -INFINITY, s = 0.0f, lse = -INFINITY;
    const float c = kLog2e / d.tau;
    if (w != 0.0f) {
        teacher(d, static_cast<const TI*>(a.ids), static_cast<const TT*>(a.t), row, id, p, sh, tm, ts);
        if (MODE == 1) {
            lse = a.lse_in[row];
        } else {
            for (int64_t v = threadIdx.x; v < d.V; v += DT) m = fmaxf(m, load_f(z, v));
            m = block_max(m, sh);
            if (m == -INFINITY) {
                float nan = 0.0f;                      // a NaN does not show in the maximum
                for (int64_t v = threadIdx.x; v < d.V; v += DT) nan += load_f(z, v) == -INFINITY ? 0.0f : load_f(z, v);
                s = block_sum(nan, sh);
                lse = s == 0.0f ? -INFINITY : NAN;
            } else {
                for (int64_t v = threadIdx.x; v < d.V; v += DT) s += exp2f((load_f(z, v) - m) * c);
                s = block_sum(s, sh);
                lse = m / d.tau + logf(s);
            }
        }
    }
    const bool empty = w == 0.0f || ts == 0.0f || lse == -INFINITY;
    if (MODE != 1) {
        float l = 0.0f;
        if (!empty)
            for (int k = threadIdx.x; k < d.K; k += DT)
                if (id[k] >= 0 && p[k] != -INFINITY) {
                    const float lp = (p[k] - tm) / d.tau, pk = exp2f((p[k] - tm) * c) / ts;
                    if (pk != 0.0f) l += pk * (lp - logf(ts) - (load_f(z, id[k]) - m) / d.tau + logf(s));
                }
        l = block_sum(l, sh);
        if (threadIdx.x == 0) {
            a.loss[row] = empty ? 0.0f : w * d.tau * d.tau * l;
            if (MODE == 0) a.lse[row] = w == 0.0f ? 0.0f : lse;
        }
    }
    if (MODE == 0) return;
    const float f = empty ? 0.0f : w * d.tau * (MODE == 1 ? a.dloss[row] : 1.0f);
    auto q = [&](int64_t v) {
        const float zv = load_f(z, v);
        return MODE == 1 ? exp2f((zv / d.tau - lse) * kLog2e) : exp2f((zv - m) * c) / s;
    };
    for (int64_t v = threadIdx.x; v < d.V; v += DT) {
        const float o = empty ? 0.0f : f * q(v);
        if constexpr (sizeof(TG) == 4) dz[v] = o;
        else dz[v] = f2bf(o);
    }
    if (empty) return;
    __syncthreads();
    // the teacher's entries again, now with their p taken off; of equal ids
    // the first writes
    for (int k = threadIdx.x; k < d.K; k += DT) {
        if (id[k] < 0) continue;
        float sum = 0.0f;
        bool first = true;
        for (int j = 0; j < d.K; ++j) {
            if (id[j] != id[k]) continue;
            first = first && j >= k;
            if (p[j] != -INFINITY) sum += exp2f((p[j] - tm) * c) / ts;
        }
        if (!first) continue;
        const float o = f * (q(id[k]) - sum);
        if constexpr (sizeof(TG) == 4) dz[id[k]] = o;
        else dz[id[k]] = f2bf(o);
    }
}

template <int MODE, typename TS, typename TG, typename TT, typename TI>
hipError_t run_t(const kan_distill_desc_t& d, const DistillArgs& a, hipStream_t s) {
    hipLaunchKernelGGL((distill_kernel<TS, TG, TT, TI, MODE>), dim3((unsigned)d.N), dim3(DT), 0, s, d, a);
    return hipGetLastError();
}
template <int MODE, typename TS, typename TG, typename TT>
hipError_t run_i(const kan_distill_desc_t& d, const DistillArgs& a, hipStream_t s) {
    return d.id_dtype == KAN_I32 ? run_t<MODE, TS, TG, TT, int32_t>(d, a, s)
                                 : run_t<MODE, TS, TG, TT, int64_t>(d, a, s);
}
template <int MODE, typename TS, typename TG>
hipError_t run_k(const kan_distill_desc_t& d, const DistillArgs& a, hipStream_t s) {
    return d.teacher_dtype == KAN_F32 ? run_i<MODE, TS, TG, float>(d, a, s) : run_i<MODE, TS, TG, uint16_t>(d, a, s);
}
template <int MODE, typename TS>
hipError_t run_g(const kan_distill_desc_t& d, const DistillArgs& a, hipStream_t s) {
    return MODE == 0 || d.grad_dtype == KAN_F32 ? run_k<MODE, TS, float>(d, a, s)
                                                : run_k<MODE, TS, uint16_t>(d, a, s);
}
template <int MODE>
hipError_t run(const kan_distill_desc_t& d, const DistillArgs& a, hipStream_t s) {
    return d.dtype == KAN_F32 ? run_g<MODE, float>(d, a, s) : run_g<MODE, uint16_t>(d, a, s);
}

}  // namespace

hipError_t launch_distill(const kan_distill_desc_t& d, const DistillPlan&, const DistillArgs& a, char*,
                          hipStream_t s) {
    return a.dz ? run<2>(d, a, s) : run<0>(d, a, s);
}

hipError_t launch_distill_bwd(const kan_distill_desc_t& d, const DistillArgs& a, hipStream_t s) {
    return run<1>(d, a, s);
}

}  // namespace kan
