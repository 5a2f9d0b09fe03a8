// Distillation from a teacher's top logits (gfx950): with p the softmax of a
// row's K teacher logits t / tau and q that of its V student logits z / tau,
//
//     loss = w tau^2 sum_k p_k (log p_k - log q_{id_k})
//     dz_v = dloss w tau (q_v - sum over k with id_k = v of p_k).
//
// K is small beside V: reading z once and writing dz once is the work, so HBM
// traffic bounds it; the arithmetic is one or two exponentials and about six
// operations an element.  Measured: step of 8192 x 65536 float32 760 us (4.1 GB,
// 5.4 TB/s), backward of 4096 x 50021 bf16 156 us (784 MB, 5.0 TB/s), forward of
// 4096 x 50021 float32 124 us (820 MB read, 6.6 TB/s).  A row's maximum m and
// s = sum exp((z - m) / tau) are kept, not their sum in lse: the loss is formed
// from z_{id} - m and log s, which are small where lse and z / tau may be large.
//
// A block takes a row.  In a step it holds the row in registers (up to 16
// vectors of 16 bytes a thread, 256 KB for 1024 threads; what is left of a
// longer row is read again from the caches), so z is read once though its
// gradient needs m and s first; the forward streams the row with a running
// maximum and sum.  The step does the teacher's part while the row's loads are
// in flight.  Its stores are plain: streamed ones gained 2% at 8192 x 65536
// and lost 4% at 4096 x 50021.
//
// The teacher's p are taken off at K of the row's elements.  Every element is
// stored by one thread, which stores it a second time where a teacher's entry
// has it: a store of another thread after a barrier may land before the first
// one, since a barrier waits for LDS but not for stores in flight.
#include "kan_distill_rows.h"
#include "kan_token.h"
#include "kan_vec.h"

namespace kan {

namespace {

constexpr float kLog2e = 1.44269504088896340736f;
// 2^x by the hardware's instruction; results below 2^-126 become 0, which no sum
// here would see.
__device__ __forceinline__ float exp2_raw(float x) { return __builtin_amdgcn_exp2f(x); }

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

// LDS of a row's teacher: ids (-1: absent) and p of its entries, and a table of
// the ids that occur, twice as large as a block has entries: the id of a slot,
// how many entries have it, and the first of them.  Then, for each thread, the
// entries whose elements it stores: the first one (-1: none), the one after
// entry k, and its gradient.  The latter two take the table's ids' place.
template <int NT>
struct TeacherShared {
    int ids[NT];
    float ps[NT];
    union {
        int key[2 * NT];
        struct {
            int next[NT];
            float value[NT];
        };
    };
    int count[2 * NT], first[2 * NT];
    int given[NT];
    float slots[3 * (NT / 64)];
};

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
    // ids and p of the row to LDS, p in place; TABLE: an empty table of ids
    template <bool TABLE>
    __device__ __forceinline__ void finish(const kan_distill_desc_t& d, TeacherShared<NT>& sh) {
        const float m = block_max<NT>(t, sh.slots);    // a NaN shows in the sum
        t = (t - (m == -INFINITY ? 0.0f : m)) / d.tau;
        p = id >= 0 ? exp2_raw(t * kLog2e) : 0.0f;
        float none = 0.0f;
        sum = p;
        block_sum2<NT>(sum, none, sh.slots + NT / 64);
        p = id >= 0 ? p / sum : 0.0f;
        sh.ids[threadIdx.x] = id;
        sh.ps[threadIdx.x] = p;
        if (TABLE) {
            sh.given[threadIdx.x] = -1;
#pragma unroll
            for (int i = threadIdx.x; i < 2 * NT; i += NT) sh.key[i] = -1, sh.count[i] = 0, sh.first[i] = NT;
        }
        __syncthreads();
    }
    // p becomes the sum over the entries of the same id, at the first of them;
    // the others drop out (id -1).  The table finds the ids that occur more than
    // once, whose entries alone are gone through (a comparison of every pair
    // took 4 us a row with 256 entries).
    __device__ __forceinline__ void join_equal(const kan_distill_desc_t& d, TeacherShared<NT>& sh) {
        int slot = 0;
        if (id >= 0) {
            slot = (int)(((uint32_t)id * 2654435769u) >> 16) & (2 * NT - 1);
            for (;;) {                                 // ends: at most NT ids in 2 NT slots
                const int was = atomicCAS(&sh.key[slot], -1, id);
                if (was == -1 || was == id) break;
                slot = (slot + 1) & (2 * NT - 1);
            }
            atomicAdd(&sh.count[slot], 1);
            atomicMin(&sh.first[slot], (int)threadIdx.x);
        }
        __syncthreads();
        if (id < 0 || sh.count[slot] == 1) return;
        if (sh.first[slot] == (int)threadIdx.x) {
            p = 0.0f;
            for (int j = 0; j < d.K; ++j) p += sh.ids[j] == id ? sh.ps[j] : 0.0f;
        } else {
            id = -1;
        }
    }
    // After join_equal: this entry's element, whose gradient is `value`, to the
    // thread that stores the element.
    __device__ __forceinline__ void give(TeacherShared<NT>& sh, int owner, float value) {
        sh.value[threadIdx.x] = value;
        sh.next[threadIdx.x] = atomicExch(&sh.given[owner], (int)threadIdx.x);
    }
};

__device__ __forceinline__ void put1(float* p, float v) { *p = v; }
__device__ __forceinline__ void put1(uint16_t* p, float v) { *p = f2bf(v); }

// What this thread was given, a barrier after the block's last `give`: over its
// own earlier stores.  The elements of a list differ, so its order is free.
template <typename TG, int NT>
__device__ __forceinline__ void put_given(TG* dz, const TeacherShared<NT>& sh) {
    for (int k = sh.given[threadIdx.x]; k >= 0; k = sh.next[k]) put1(dz + sh.ids[k], sh.value[k]);
}

template <typename TS, int N>
__device__ __forceinline__ float max_of(const Raw<TS, N>& r) {
    float m = raw_value(r, 0);
#pragma unroll
    for (int i = 1; i < N; ++i) m = fmaxf(m, raw_value(r, i));
    return m;
}

constexpr int VE = 4;             // elements of a vector (backward between bf16 arrays: 8)

// All of a row's gradient, or of its elements [v0, v1), zero.
template <typename TG, int NT>
__device__ __forceinline__ void zeros(TG* dz, int64_t v0, int64_t v1) {
    const float zero[VE] = {};
    dz += v0;
    const int64_t n = v1 - v0;
    const int head = head_of(dz, n);
    const int64_t tail = n - (n - head) % VE;
    for (int64_t v = head + (int64_t)threadIdx.x * VE; v + VE <= n; v += NT * VE) store_vec<VE>(dz + v, zero);
    for (int v = threadIdx.x; v < head; v += NT) put1(dz + v, 0.0f);
    if (tail + threadIdx.x < n) put1(dz + tail + threadIdx.x, 0.0f);
}

// Forward (STEP false) and step.  NV vectors of a thread are held in registers.
template <typename TS, typename TG, int NT, int NV, bool STEP, bool STREAM>
__global__ void __launch_bounds__(NT) distill_row_kernel(kan_distill_desc_t d, DistillArgs a) {
    constexpr int W = NT / 64;
    typedef Raw<TS, VE> Vec;
    __shared__ TeacherShared<NT> sh;
    __shared__ float slots[3 * W];
    const int64_t row = blockIdx.x, V = d.V;
    const TS* z = static_cast<const TS*>(a.z) + row * d.z_row;
    TG* dz = STEP ? static_cast<TG*>(a.dz) + row * d.dz_row : nullptr;
    const float w = a.w ? a.w[row] : 1.0f;
    if (STEP && w == 0.0f) {                           // the forward's lse is due for every row
        if (threadIdx.x == 0) a.loss[row] = 0.0f;
        zeros<TG, NT>(dz, 0, V);
        return;
    }
    const float inv = 1.0f / d.tau, c = kLog2e * inv;
    Teacher<NT> te;
    te.load(d, a, row);
    const int head = STEP ? head_of(dz, V) : head_of(z, V);
    const int64_t body = head + (int64_t)threadIdx.x * VE, tail = V - (V - head) % VE + threadIdx.x;
    constexpr int64_t STRIDE = NT * VE;                // elements of a vector of every thread
    float hz = -INFINITY, tz = -INFINITY;
    if ((int)threadIdx.x < head) hz = load_f(z, threadIdx.x);
    if (tail < V) tz = load_f(z, tail);
    Vec keep[NV ? NV : 1];
    float m = -INFINITY, s = 0.0f;
    if (NV) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (head + v * STRIDE >= V) break;         // uniform
            if (body + v * STRIDE + VE <= V) {
                keep[v] = load_raw<TS, VE>(z + body + v * STRIDE);
            } else {
#pragma unroll
                for (int i = 0; i < Vec::W; ++i) keep[v].w[i] = sizeof(TS) == 4 ? 0xff800000u : 0xff80ff80u;
            }
        }
    }
    te.template finish<STEP>(d, sh);
    // a running maximum and sum over what registers do not hold
    for (int64_t v = body + NV * STRIDE; v + VE <= V; v += STRIDE * DU) {
        Vec q[DU];
#pragma unroll
        for (int u = 0; u < DU; ++u) {
            const int64_t at = v + u * STRIDE;         // past the end: the first again, not counted
            const TS* from = z + (at + VE <= V ? at : v);
            q[u] = STREAM ? load_once<TS, VE>(from) : load_raw<TS, VE>(from);
        }
        float g = m;
#pragma unroll
        for (int u = 0; u < DU; ++u) g = fmaxf(g, max_of<TS, VE>(q[u]));
        const float g0 = g == -INFINITY ? 0.0f : g;
        s *= exp2_raw((m - g0) * c);
        m = g;
#pragma unroll
        for (int u = 0; u < DU; ++u) {
            if (v + u * STRIDE + VE > V) continue;
#pragma unroll
            for (int i = 0; i < VE; ++i) s += exp2_raw((raw_value(q[u], i) - g0) * c);
        }
    }
    const float m_stream = m;
    m = fmaxf(m, fmaxf(hz, tz));
    if (NV) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (head + v * STRIDE >= V) break;
            m = fmaxf(m, max_of<TS, VE>(keep[v]));
        }
    }
    m = block_max<NT>(m, slots);
    const float m0 = m == -INFINITY ? 0.0f : m;
    s *= exp2_raw((m_stream - m0) * c);
    hz = exp2_raw((hz - m0) * c);
    tz = exp2_raw((tz - m0) * c);
    s += hz + tz;
    if (NV) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (head + v * STRIDE >= V) break;
#pragma unroll
            for (int i = 0; i < VE; ++i) {
                const float e = exp2_raw((raw_value(keep[v], i) - m0) * c);
                s += e;
                if constexpr (STEP && sizeof(TS) == 4) keep[v].w[i] = __float_as_uint(e);
            }
        }
    }
    // sum_k p_k (log p_k + log(teacher's sum) - (z_k - m) / tau); the logs of the sums come after it
    float l = 0.0f, zk = -INFINITY;
    if (te.id >= 0) {
        zk = load_f(z, te.id);
        if (te.p != 0.0f) l = te.p * (te.t - (zk - m0) * inv);
    }
    if (STEP) te.join_equal(d, sh);
    block_sum2<NT>(s, l, slots + W);
    const bool empty = w == 0.0f || te.sum == 0.0f || s == 0.0f;
    if (threadIdx.x == 0) {
        a.loss[row] = empty ? 0.0f : w * d.tau * d.tau * (l - logf(te.sum) + logf(s));
        if (!STEP) a.lse[row] = m0 * inv + logf(s);
    }
    if (!STEP) return;
    if (empty) {
        zeros<TG, NT>(dz, 0, V);
        return;
    }
    const float f = w * d.tau, fs = f / s;
    if (te.id >= 0) te.give(sh, owner_of(te.id, head, V, VE, NT), fs * exp2_raw((zk - m0) * c) - f * te.p);
    if ((int)threadIdx.x < head) put1(dz + threadIdx.x, fs * hz);
    if (tail < V) put1(dz + tail, fs * tz);
    if (NV) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (head + v * STRIDE >= V) break;
            if (body + v * STRIDE + VE > V) break;
            float o[VE];
#pragma unroll
            for (int i = 0; i < VE; ++i) {
                const float e = raw_value(keep[v], i);
                o[i] = fs * (sizeof(TS) == 4 ? e : exp2_raw((e - m0) * c));
            }
            store_vec<VE>(dz + body + v * STRIDE, o);
        }
    }
    for (int64_t v = body + NV * STRIDE; v + VE <= V; v += STRIDE * DU) {
        Vec q[DU];
#pragma unroll
        for (int u = 0; u < DU; ++u) {
            const int64_t at = v + u * STRIDE;
            q[u] = load_raw<TS, VE>(z + (at + VE <= V ? at : v));
        }
#pragma unroll
        for (int u = 0; u < DU; ++u) {
            if (v + u * STRIDE + VE > V) continue;
            float o[VE];
#pragma unroll
            for (int i = 0; i < VE; ++i) o[i] = fs * exp2_raw((raw_value(q[u], i) - m0) * c);
            store_vec<VE>(dz + v + u * STRIDE, o);
        }
    }
    __syncthreads();
    put_given<TG, NT>(dz, sh);
}

// Maximum and sum of exp((z - max) / tau) of part p of a row, for a step of few
// long rows: out[row][p].
template <typename TS, int NT>
__global__ void __launch_bounds__(NT) distill_part_kernel(kan_distill_desc_t d, DistillArgs a, int parts, int64_t part,
                                                          float2* out) {
    __shared__ float slots[3 * (NT / 64)];
    const int64_t row = blockIdx.x / (unsigned)parts, V = d.V;
    const int p = (int)(blockIdx.x % (unsigned)parts);
    if (a.w && a.w[row] == 0.0f) return;               // not read in the second launch
    const TS* z = static_cast<const TS*>(a.z) + row * d.z_row;
    const int head = head_of(z, V);
    const Part at(p, part, head, V, VE);
    const float c = kLog2e / d.tau;
    constexpr int64_t STRIDE = NT * VE;
    float m = -INFINITY, s = 0.0f;
    const float hz = p == 0 && (int)threadIdx.x < head ? load_f(z, threadIdx.x) : -INFINITY;
    const float tz = at.tail + threadIdx.x < V ? load_f(z, at.tail + threadIdx.x) : -INFINITY;
    for (int64_t v = at.v + (int64_t)threadIdx.x * VE; v + VE <= at.v1; v += STRIDE * DU) {
        Raw<TS, VE> q[DU];
#pragma unroll
        for (int u = 0; u < DU; ++u) {
            const int64_t e = v + u * STRIDE;
            q[u] = load_raw<TS, VE>(z + (e + VE <= at.v1 ? e : v));
        }
        float g = m;
#pragma unroll
        for (int u = 0; u < DU; ++u) g = fmaxf(g, max_of<TS, VE>(q[u]));
        const float g0 = g == -INFINITY ? 0.0f : g;
        s *= exp2_raw((m - g0) * c);
        m = g;
#pragma unroll
        for (int u = 0; u < DU; ++u) {
            if (v + u * STRIDE + VE > at.v1) continue;
#pragma unroll
            for (int i = 0; i < VE; ++i) s += exp2_raw((raw_value(q[u], i) - g0) * c);
        }
    }
    const float mine = m;
    m = block_max<NT>(fmaxf(m, fmaxf(hz, tz)), slots);
    const float m0 = m == -INFINITY ? 0.0f : m;
    s = s * exp2_raw((mine - m0) * c) + exp2_raw((hz - m0) * c) + exp2_raw((tz - m0) * c);
    float none = 0.0f;
    block_sum2<NT>(s, none, slots + NT / 64);
    if (threadIdx.x == 0) out[blockIdx.x] = make_float2(m, s);
}

// Backward, or (STEP) the second launch of a step of few long rows: block (row,
// p) writes part p of a row's gradient; a step's first block the loss too.
template <typename TS, typename TG, int NT, int VE, bool STREAM, bool STEP>
__global__ void __launch_bounds__(NT) distill_bwd_kernel(kan_distill_desc_t d, DistillArgs a, int parts, int64_t part,
                                                         const float2* sums, int n_sums) {
    __shared__ TeacherShared<NT> sh;
    __shared__ float slots[2 * (NT / 64)];
    const int64_t row = blockIdx.x / (unsigned)parts, V = d.V;
    const int p = (int)(blockIdx.x % (unsigned)parts);
    const TS* z = static_cast<const TS*>(a.z) + row * d.z_row;
    TG* dz = static_cast<TG*>(a.dz) + row * d.dz_row;
    const int head = head_of(dz, V);
    const Part at(p, part, head, V, VE);
    const float w = a.w ? a.w[row] : 1.0f, inv = 1.0f / d.tau, c = kLog2e * inv;
    float lse = 0.0f, m0 = 0.0f, s = 0.0f;
    bool empty = w == 0.0f;
    if (!empty && STEP) {
        // every wave joins the parts' sums, a lane to a part (at most 64)
        const int lane = threadIdx.x & 63;
        const float2 q = lane < n_sums ? sums[row * n_sums + lane] : make_float2(-INFINITY, 0.0f);
        float m = q.x;
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
        m0 = m == -INFINITY ? 0.0f : m;
        s = q.y * exp2_raw((q.x - m0) * c);
        if (q.y == 0.0f) s = 0.0f;                     // a part of -inf only
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) s += __shfl_xor(s, o, 64);
        empty = s == 0.0f;
    } else if (!empty) {
        lse = a.lse_in[row];
        empty = lse == -INFINITY;
    }
    Teacher<NT> te;
    if (!empty) {                                      // uniform across the block
        te.load(d, a, row);
        te.template finish<true>(d, sh);
        empty = te.sum == 0.0f;
    }
    if (empty) {
        zeros<TG, NT>(dz, at.v0, at.v1);
        if (STEP && p == 0 && threadIdx.x == 0) a.loss[row] = 0.0f;
        return;
    }
    if (STEP && p == 0) {
        float l = 0.0f, none = 0.0f;
        if (te.id >= 0 && te.p != 0.0f) l = te.p * (te.t - (load_f(z, te.id) - m0) * inv);
        block_sum2<NT>(l, none, slots);
        if (threadIdx.x == 0) a.loss[row] = w * d.tau * d.tau * (l - logf(te.sum) + logf(s));
    }
    const bool here = te.id >= at.v0 && te.id < at.v1;
    const float zk = here ? load_f(z, te.id) : 0.0f;
    te.join_equal(d, sh);
    const float f = w * d.tau * (STEP ? 1.0f : a.dloss[row]), fs = STEP ? f / s : f;
    auto fq = [&](float x) {                           // f q
        return fs * exp2_raw(STEP ? (x - m0) * c : __builtin_fmaf(x, inv, -lse) * kLog2e);
    };
    if (here && te.id >= 0) te.give(sh, owner_of(te.id, head, V, VE, NT), fq(zk) - f * te.p);
    constexpr int64_t STRIDE = NT * VE;
    for (int64_t v = at.v + (int64_t)threadIdx.x * VE; v + VE <= at.v1; v += STRIDE * DU) {
        Raw<TS, VE> x[DU];
#pragma unroll
        for (int u = 0; u < DU; ++u) {
            const int64_t e = v + u * STRIDE;
            x[u] = load_raw<TS, VE>(z + (e + VE <= at.v1 ? e : v));
        }
#pragma unroll
        for (int u = 0; u < DU; ++u) {
            if (v + u * STRIDE + VE > at.v1) continue;
            float o[VE];
#pragma unroll
            for (int i = 0; i < VE; ++i) o[i] = fq(raw_value(x[u], i));
            store_vec<VE, STREAM>(dz + v + u * STRIDE, o);
        }
    }
    if (p == 0 && (int)threadIdx.x < head) put1(dz + threadIdx.x, fq(load_f(z, threadIdx.x)));
    const int64_t tail = at.tail + threadIdx.x;
    if (tail < V) put1(dz + tail, fq(load_f(z, tail)));
    __syncthreads();
    put_given<TG, NT>(dz, sh);
}

template <typename TS, typename TG, int NT, int NV, bool STEP, bool STREAM>
hipError_t row_t(const kan_distill_desc_t& d, const DistillArgs& a, hipStream_t s) {
    hipLaunchKernelGGL((distill_row_kernel<TS, TG, NT, NV, STEP, STREAM>), dim3((unsigned)d.N), dim3(NT), 0, s, d, a);
    return hipGetLastError();
}

// The fewest threads whose registers hold a row, and at least one for each of
// the teacher's entries.
template <typename TS, typename TG>
hipError_t step_t(const kan_distill_desc_t& d, const DistillArgs& a, hipStream_t s) {
    constexpr int NV = 256 / (VE * (int)sizeof(TS));   // 64 registers
    constexpr int64_t per = NV * VE;
    const int64_t threads = std::max((d.V + per - 1) / per, d.K);
    // short rows leave most of the registers free, and their time is latency:
    // more of them at a time (16384 x 4000 bf16 129 -> 88 us, 16384 x 3000 float32
    // 121 -> 85)
    if (d.K <= 64 && 4 * d.V <= 64 * per) return row_t<TS, TG, 64, NV / 4, true, false>(d, a, s);
    if (d.K <= 256 && 4 * d.V <= 256 * per) return row_t<TS, TG, 256, NV / 4, true, false>(d, a, s);
    if (threads <= 256) return row_t<TS, TG, 256, NV, true, false>(d, a, s);
    if (threads <= 512) return row_t<TS, TG, 512, NV, true, false>(d, a, s);
    return row_t<TS, TG, 1024, NV, true, false>(d, a, s);
}

// Few long rows take a block of 1024 threads each (64 x 131072 float32: 16 us, 31
// with 256), many rows one of 256 (16384 x 4000 bf16, K = 128: 45 us, 84 with 512),
// short ones with few teacher's logits a wave (K = 64: 32 us, 43 with 256).
template <typename TS, bool STREAM>
hipError_t fwd_s(const kan_distill_desc_t& d, const DistillArgs& a, hipStream_t s) {
    if (d.K > 256 || (d.N <= 512 && d.V >= 8192)) return row_t<TS, TS, 1024, 0, false, STREAM>(d, a, s);
    if (d.K > 64 || d.V > 64 * 64) return row_t<TS, TS, 256, 0, false, STREAM>(d, a, s);
    return row_t<TS, TS, 64, 0, false, STREAM>(d, a, s);
}
// Past kStreamBytes the logits cannot stay in the caches for the backward pass
// and are read as streamed data (4096 x 50021: float32 141 -> 124 us, bf16 76 -> 69).
template <typename TS>
hipError_t fwd_t(const kan_distill_desc_t& d, const DistillArgs& a, hipStream_t s) {
    return d.N * d.V * (int64_t)sizeof(TS) >= kStreamBytes ? fwd_s<TS, true>(d, a, s) : fwd_s<TS, false>(d, a, s);
}

template <typename TS, typename TG, int NT, bool STEP>
hipError_t bwd_n(const kan_distill_desc_t& d, const DistillArgs& a, const float2* sums, int n_sums, hipStream_t s) {
    constexpr int VE = sizeof(TS) == 2 && sizeof(TG) == 2 ? 8 : 4;     // 16 bytes of the wider type
    constexpr int64_t round = NT * VE;
    // Blocks of one round of loads each, up to 32768 of them: 4096 x 50021 takes
    // 181 us (bf16) and 348 us (float32) with a block to a row, 163 and 319 cut (all
    // of these on one card; another one took 156).
    const int64_t parts = std::max<int64_t>(1, std::min<int64_t>((32768 + d.N - 1) / d.N, d.V / (round * DU)));
    const int64_t part = round_up((d.V + parts - 1) / parts, round), n = (d.V + part - 1) / part;
    const dim3 grid((unsigned)(d.N * n));
    // streamed stores past kStreamBytes: 4096 x 50021 bf16 166 -> 163 us, float32
    // 322 -> 319, and 197 -> 170 and 372 -> 331 with a block to a row (a step of few
    // rows does not come near)
    if (!STEP && d.N * d.V * (int64_t)sizeof(TG) >= kStreamBytes)
        hipLaunchKernelGGL((distill_bwd_kernel<TS, TG, NT, VE, !STEP, STEP>), grid, dim3(NT), 0, s, d, a, (int)n, part,
                           sums, n_sums);
    else
        hipLaunchKernelGGL((distill_bwd_kernel<TS, TG, NT, VE, false, STEP>), grid, dim3(NT), 0, s, d, a, (int)n, part,
                           sums, n_sums);
    return hipGetLastError();
}
template <typename TS, typename TG, bool STEP>
hipError_t bwd_t(const kan_distill_desc_t& d, const DistillArgs& a, const float2* sums, int n_sums, hipStream_t s) {
    if (d.K > 256) return bwd_n<TS, TG, 1024, STEP>(d, a, sums, n_sums, s);
    if (STEP || d.K > 64 || d.V > 64 * 64) return bwd_n<TS, TG, 256, STEP>(d, a, sums, n_sums, s);
    return bwd_n<TS, TG, 64, STEP>(d, a, sums, n_sums, s);
}

template <typename TS, typename TG>
hipError_t cut_step(const kan_distill_desc_t& d, const DistillPlan& p, const DistillArgs& a, char* ws, hipStream_t s) {
    float2* sums = reinterpret_cast<float2*>(ws);
    hipLaunchKernelGGL((distill_part_kernel<TS, 256>), dim3((unsigned)(d.N * p.parts)), dim3(256), 0, s, d, a, p.parts,
                       p.part, sums);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess ? e : bwd_t<TS, TG, true>(d, a, sums, p.parts, s);
}

template <typename TS, typename TG>
hipError_t step(const kan_distill_desc_t& d, const DistillPlan& p, const DistillArgs& a, char* ws, hipStream_t s) {
    return p.parts > 1 ? cut_step<TS, TG>(d, p, a, ws, s) : step_t<TS, TG>(d, a, s);
}

}  // namespace

hipError_t launch_distill(const kan_distill_desc_t& d, const DistillPlan& p, const DistillArgs& a, char* ws,
                          hipStream_t s) {
    if (!a.dz) return d.dtype == KAN_F32 ? fwd_t<float>(d, a, s) : fwd_t<uint16_t>(d, a, s);
    if (d.dtype == KAN_F32)
        return d.grad_dtype == KAN_F32 ? step<float, float>(d, p, a, ws, s) : step<float, uint16_t>(d, p, a, ws, s);
    return d.grad_dtype == KAN_F32 ? step<uint16_t, float>(d, p, a, ws, s) : step<uint16_t, uint16_t>(d, p, a, ws, s);
}

hipError_t launch_distill_bwd(const kan_distill_desc_t& d, const DistillArgs& a, hipStream_t s) {
    if (d.dtype == KAN_F32)
        return d.grad_dtype == KAN_F32 ? bwd_t<float, float, false>(d, a, nullptr, 0, s)
                                       : bwd_t<float, uint16_t, false>(d, a, nullptr, 0, s);
    return d.grad_dtype == KAN_F32 ? bwd_t<uint16_t, float, false>(d, a, nullptr, 0, s)
                                   : bwd_t<uint16_t, uint16_t, false>(d, a, nullptr, 0, s);
}

}  // namespace kan
