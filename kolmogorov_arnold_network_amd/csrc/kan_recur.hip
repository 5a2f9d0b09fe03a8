// Gated linear recurrence over the rows of a sequence, each channel on its own
// (gfx950):
//
//     u_t = sigmoid(-g_t),  h_t = h_{t-1} + u_t (x_t - h_{t-1})
//
// its backward pass, and its single-row step on a pool of states.
//
// A step is taken from the side that the gate is near, by the smaller of the
// two shares s = min(u, f): h + u (x - h) where f >= u, x + f (h - x) otherwise.
// A share that rounds to 1 has lost the digits of the other one, which decide
// how long a memory is (f near 1) or how much of a large state is left (u near
// 1).  Backward, with c_t = f_t del_t the gradient that row t hands to row t - 1
// (c_len = dhT), in the same way:
//
//     del_t = dy_t + c_{t+1},  c_t = del_t - u_t del_t (f >= u), f_t del_t,
//     dx_t = u_t del_t,  dg_t = f_t u_t (h_{t-1} - x_t) del_t,  dh0 = c_0.
#include "kan_token.h"
#include "kan_vec.h"

namespace kan {

namespace {

// The shares of x (u = sigmoid(-g)) and of the state (f = sigmoid(g)), each to
// a few ulp of its own size: the smaller one, the larger one, and whether the
// state's is the larger.
struct Gate {
    float s, l;
    bool keep;
    __device__ __forceinline__ explicit Gate(float g) {
        const float e = __expf(-fabsf(g));
        l = __builtin_amdgcn_rcpf(1.0f + e);
        s = e * l;
        keep = g >= 0.0f;
    }
    __device__ __forceinline__ float u() const { return keep ? s : l; }
    __device__ __forceinline__ float step(float h, float x) const {
        const float a = keep ? h : x, b = keep ? x : h;
        return __builtin_fmaf(s, b - a, a);
    }
    __device__ __forceinline__ float back(float del) const {
        return __builtin_fmaf(keep ? -s : s, del, keep ? del : 0.0f);
    }
};

__device__ __forceinline__ int64_t length_of(const int32_t* lengths, int64_t b, int64_t T) {
    return lengths ? min(max((int64_t)lengths[b], (int64_t)0), T) : T;
}

// The sequence and the channel of a thread (64 channels of a sequence to a block).
__device__ __forceinline__ bool channel(const kan_recur_desc_t& d, int64_t& b, int64_t& c) {
    const unsigned cb = (unsigned)((d.D + 63) / 64);
    b = blockIdx.x / cb;
    c = (int64_t)(blockIdx.x % cb) * 64 + threadIdx.x;
    return c < d.D;
}

template <typename TS>
__global__ void __launch_bounds__(64) recur_fwd_kernel(kan_recur_desc_t d, RecurArgs a) {
    int64_t b, c;
    if (!channel(d, b, c)) return;
    const int64_t len = length_of(a.lengths, b, d.T);
    const TS* x = static_cast<const TS*>(a.x) + b * d.x_seq + c;
    const TS* g = static_cast<const TS*>(a.g) + b * d.g_seq + c;
    float* y = a.out + b * d.T * d.D + c;
    float h = a.h0 ? a.h0[b * d.D + c] : 0.0f;
    for (int64_t t = 0; t < len; ++t) {
        h = Gate(load_f(g, t * d.g_row)).step(h, load_f(x, t * d.x_row));
        y[t * d.D] = h;
    }
    for (int64_t t = len; t < d.T; ++t) y[t * d.D] = 0.0f;
    if (a.hT) a.hT[b * d.D + c] = h;
}

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t* p, float v) { *p = f2bf(v); }

template <typename TS, typename TG>
__global__ void __launch_bounds__(64) recur_bwd_kernel(kan_recur_desc_t d, RecurArgs a) {
    int64_t b, c;
    if (!channel(d, b, c)) return;
    const int64_t len = length_of(a.lengths, b, d.T);
    const TS* x = static_cast<const TS*>(a.x) + b * d.x_seq + c;
    const TS* g = static_cast<const TS*>(a.g) + b * d.g_seq + c;
    const float* y = a.y + b * d.T * d.D + c;
    const float* dy = a.dy + b * d.T * d.D + c;
    TG* dx = a.dx ? static_cast<TG*>(a.dx) + b * d.dx_seq + c : nullptr;
    TG* dg = a.dx ? static_cast<TG*>(a.dg) + b * d.dg_seq + c : nullptr;
    float k = a.dhT ? a.dhT[b * d.D + c] : 0.0f;
    if (dx)
        for (int64_t t = len; t < d.T; ++t) put(dx + t * d.dx_row, 0.0f), put(dg + t * d.dg_row, 0.0f);
    for (int64_t t = len - 1; t >= 0; --t) {
        const Gate q(load_f(g, t * d.g_row));
        const float del = dy[t * d.D] + k;
        if (dx) {
            const float before = t > 0 ? y[(t - 1) * d.D] : a.h0 ? a.h0[b * d.D + c] : 0.0f;
            put(dx + t * d.dx_row, q.u() * del);
            put(dg + t * d.dg_row, q.s * q.l * (before - load_f(x, t * d.x_row)) * del);
        }
        k = q.back(del);
    }
    if (a.dh0) a.dh0[b * d.D + c] = k;
}

template <typename TS>
__global__ void __launch_bounds__(64) recur_step_kernel(kan_recur_desc_t d, int64_t S, const TS* x, const TS* g,
                                                        float* state, const int32_t* slots, float* y) {
    int64_t b, c;
    if (!channel(d, b, c)) return;
    const int64_t slot = slots ? (int64_t)slots[b] : b;
    if (slot < 0 || slot >= S) {
        y[b * d.D + c] = 0.0f;
        return;
    }
    float* st = state + slot * d.D + c;
    const float n = Gate(load_f(g, b * d.g_seq + c)).step(*st, load_f(x, b * d.x_seq + c));
    *st = n;
    y[b * d.D + c] = n;
}

dim3 channel_grid(const kan_recur_desc_t& d) { return dim3((unsigned)((d.D + 63) / 64 * d.B)); }

}  // namespace

hipError_t launch_recur_fwd(const kan_recur_desc_t& d, const RecurPlan&, const RecurArgs& a, char*, hipStream_t s) {
    if (d.dtype == KAN_F32)
        hipLaunchKernelGGL(recur_fwd_kernel<float>, channel_grid(d), dim3(64), 0, s, d, a);
    else
        hipLaunchKernelGGL(recur_fwd_kernel<uint16_t>, channel_grid(d), dim3(64), 0, s, d, a);
    return hipGetLastError();
}

hipError_t launch_recur_bwd(const kan_recur_desc_t& d, const RecurPlan&, const RecurArgs& a, char*, hipStream_t s) {
    const dim3 grid = channel_grid(d);
    if (d.dtype == KAN_F32 && d.grad_dtype == KAN_F32)
        hipLaunchKernelGGL((recur_bwd_kernel<float, float>), grid, dim3(64), 0, s, d, a);
    else if (d.dtype == KAN_F32)
        hipLaunchKernelGGL((recur_bwd_kernel<float, uint16_t>), grid, dim3(64), 0, s, d, a);
    else if (d.grad_dtype == KAN_F32)
        hipLaunchKernelGGL((recur_bwd_kernel<uint16_t, float>), grid, dim3(64), 0, s, d, a);
    else
        hipLaunchKernelGGL((recur_bwd_kernel<uint16_t, uint16_t>), grid, dim3(64), 0, s, d, a);
    return hipGetLastError();
}

hipError_t launch_recur_step(const kan_recur_desc_t& d, int64_t S, const void* x, const void* g, float* state,
                             const int32_t* slots, float* y, hipStream_t s) {
    if (d.dtype == KAN_F32)
        hipLaunchKernelGGL(recur_step_kernel<float>, channel_grid(d), dim3(64), 0, s, d, S,
                           static_cast<const float*>(x), static_cast<const float*>(g), state, slots, y);
    else
        hipLaunchKernelGGL(recur_step_kernel<uint16_t>, channel_grid(d), dim3(64), 0, s, d, S,
                           static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(g), state, slots, y);
    return hipGetLastError();
}

}  // namespace kan
