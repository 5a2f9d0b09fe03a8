// Gated delta rule (gfx950): a state S [Dk, Dv] for each head of a sequence,
//
//     S' = exp(g_t) S,  w_t = v_t - S'^T k_t,  u_t = beta_t w_t,
//     S  = S' + k_t u_t^T,  y_t = scale S^T q_t.
//
// Row by row it is two products of a vector with S; in chunks of 64 rows it is
// products of matrices.  With c_i the sum of g from the chunk's start to row i,
// D_ij = exp(c_i - c_j) and S0 the chunk's first state,
//
//     A_ij = (k_i . k_j) D_ij  (j < i),    G = (I + A diag(beta))^-1 A
//     e = V - exp(c) K S0,    w = e - G (beta e),    u = beta w
//     P_ij = scale (q_i . k_j) D_ij  (j <= i),    Y = scale exp(c) Q S0 + P u
//     S1 = exp(c_63) S0 + K^T (exp(c_63 - c) u).
//
// One launch makes the chunks' G and P (all chunks at once), a second one walks
// along the sequences with a block for 32 columns of a state.  G is kept rather
// than the inverse: both (I + A diag(beta))^-1 = I - G diag(beta) and its
// counterpart (I + diag(beta) A)^-1 = I - diag(beta) G come from it, also where
// beta is 0.  Backward, from dY and the gradient dS1 of the chunk's last state:
//
//     du = P^T dY + exp(c_63 - c) K dS1,    r = du - G^T (beta du),    dv = beta r
//     dS0 = exp(c_63) dS1 + scale Q^T exp(c) dY - K^T exp(c) dv,    dbeta = r . w
//     dP = dY u^T,   X = dv u^T  (j < i)
//     dq = scale exp(c) dY S0^T + scale (dP D) K
//     dk = scale (dP D)^T Q + exp(c_63 - c) u dS1^T - exp(c) dv S0^T
//          - (X D) K - (X D)^T K
//
// and dg_t is the sum over all that a decay at row t stands between: the pairs
// i >= t > j of (dP P - X A)_ij, the parts of rows i >= t that come from S0, those
// of rows j < t that reach dS1, and exp(c_63) <dS1, S0>.  Every one of these has
// the decay of row t in it, so that a gradient keeps its digits where decays are
// strong; sums of q . dq - k . dk over a sequence would lose them.
//
// c is kept as the sum of two floats: differences of long sums lose nothing.
#include "kan_delta.h"
#include "kan_vec.h"

namespace kan {

namespace {

constexpr int C = kDeltaChunk, NV = kDeltaTile;
constexpr int NT = 256;              // threads of a block: four waves, 16 rows of a chunk each
constexpr int LC = C + 4;            // LDS pitch of 64 floats: rows 16 bytes apart modulo the banks
constexpr float kUnitEps = 1e-6f;

typedef float f32x4 __attribute__((ext_vector_type(4)));

// What a chunk's rows have for themselves: [8][64] floats of a chunk-head.
enum RowField { kHi, kLo, kBeta, kNk, kNq, kFrom, kTo, kFields = 8 };

__device__ __forceinline__ f32x4 zero4() { return f32x4{0.0f, 0.0f, 0.0f, 0.0f}; }

// acc += A B over 16 values of the contracted index.  Lane l has A's row l % 16
// (or B's column) at the four values 4 (l / 16) .. 4 (l / 16) + 3 of the index; acc has
// rows 4 (l / 16) .. + 3 of column l % 16.
__device__ __forceinline__ void mma(f32x4& acc, const f32x4& a, const f32x4& b) {
#pragma unroll
    for (int j = 0; j < 4; ++j) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], acc, 0, 0, 0);
}
__device__ __forceinline__ f32x4 ld4(const float* p) { return *reinterpret_cast<const f32x4*>(p); }
__device__ __forceinline__ void st4(float* p, const f32x4& v) { *reinterpret_cast<f32x4*>(p) = v; }

// Elements at .. at + 3 of a row of D, zero past its end.
template <typename TS>
__device__ __forceinline__ f32x4 row4(const TS* p, int at, int D) {
    f32x4 v = zero4();
    if (at + 4 <= D) {
        const Raw<TS, 4> r = load_raw<TS, 4>(p + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = raw_value(r, i);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (at + i < D) v[i] = load_f(p, at + i);
    }
    return v;
}
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t* p, float v) { *p = f2bf(v); }

__device__ __forceinline__ int64_t at_row(const kan_heads_t& s, int64_t b, int64_t t, int64_t h) {
    return b * s.seq + t * s.row + h * s.head;
}
__device__ __forceinline__ int length_of(const DeltaArgs& a, int64_t b, int64_t T) {
    if (!a.lengths) return (int)T;
    const int n = a.lengths[b];
    return n < 0 ? 0 : n > T ? (int)T : n;
}
__device__ __forceinline__ float decay(const float* row, int i, int j) {
    return expf((row[kHi * C + i] - row[kHi * C + j]) + (row[kLo * C + i] - row[kLo * C + j]));
}

// ---- a chunk's rows among themselves -------------------------------------------

// Rows of q or k to LDS (pitch DKP + 4), zero past the length and past Dk.
template <typename TS, int DKP>
__device__ __forceinline__ void fill_rows(float* lds, const TS* base, int64_t row_stride, int rows, int Dk) {
    const int i = threadIdx.x >> 2;
#pragma unroll
    for (int s = 0; s < DKP / 16; ++s) {
        const int d = 16 * s + 4 * (threadIdx.x & 3);
        st4(lds + i * (DKP + 4) + d, i < rows ? row4<TS>(base + i * row_stride, d, Dk) : zero4());
    }
}
// Every row times its factor.
template <int DKP>
__device__ __forceinline__ void scale_rows(float* lds, const float* factor) {
    const int i = threadIdx.x >> 2;
    const float f = factor[i];
#pragma unroll
    for (int s = 0; s < DKP / 16; ++s) {
        float* p = lds + i * (DKP + 4) + 16 * s + 4 * (threadIdx.x & 3);
        st4(p, ld4(p) * f);
    }
}
template <int DKP>
__device__ __forceinline__ void unit_factors(const float* lds, float* factor) {
    const int i = threadIdx.x >> 2;
    float n = 0.0f;
#pragma unroll
    for (int s = 0; s < DKP / 16; ++s) {
        const f32x4 v = ld4(lds + i * (DKP + 4) + 16 * s + 4 * (threadIdx.x & 3));
#pragma unroll
        for (int j = 0; j < 4; ++j) n = __builtin_fmaf(v[j], v[j], n);
    }
    n += __shfl_xor(n, 1, 64);
    n += __shfl_xor(n, 2, 64);
    if ((threadIdx.x & 3) == 0) factor[i] = 1.0f / sqrtf(n + kUnitEps);
}

// Chunk n of head h of sequence b: row fields, G and P (BWD: their transposes too).
template <typename TS, int DKP, bool BWD>
__global__ void __launch_bounds__(NT) delta_prep_kernel(kan_delta_desc_t d, DeltaPlan p, DeltaArgs a, char* ws) {
    extern __shared__ float lds[];
    float* K = lds;                                    // [64][DKP + 4]
    float* Q = K + C * (DKP + 4);
    float* A = Q + C * (DKP + 4);                      // [64][LC]
    float* G = A + C * LC;
    float* row = G + C * LC;                           // [8][64]
    const int64_t n = blockIdx.x % (unsigned)p.chunks, bh = blockIdx.x / (unsigned)p.chunks;
    const int64_t b = bh / d.Hv, h = bh % d.Hv, hk = h / (d.Hv / d.Hk);
    const int rows = length_of(a, b, d.T) - (int)n * C;
    if (rows <= 0) return;                             // uniform
    const int64_t t0 = n * C;
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, r = lane & 15, gq = lane >> 4;
    fill_rows<TS, DKP>(K, static_cast<const TS*>(a.k) + at_row(d.k, b, t0, hk), d.k.row, rows, (int)d.Dk);
    fill_rows<TS, DKP>(Q, static_cast<const TS*>(a.q) + at_row(d.q, b, t0, hk), d.q.row, rows, (int)d.Dk);
    if (wave == 0) {
        float g = 0.0f, beta = 0.0f;
        if (lane < rows) {
            g = a.g[(b * d.T + t0 + lane) * d.Hv + h];
            beta = a.beta[(b * d.T + t0 + lane) * d.Hv + h];
            g = g < -128.0f ? -128.0f : g;             // exp(-128) is 0; a NaN stays
        }
        double c = g;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const double before = __shfl_up(c, o, 64);
            if (lane >= o) c += before;
        }
        const float hi = (float)c, lo = (float)(c - (double)hi);
        row[kHi * C + lane] = hi;
        row[kLo * C + lane] = hi - hi == 0.0f ? lo : 0.0f;
        row[kBeta * C + lane] = beta;
        row[kNk * C + lane] = row[kNq * C + lane] = 1.0f;
        row[kFrom * C + lane] = (float)exp(c);
        row[kTo * C + lane] = (float)exp(__shfl(c, 63, 64) - c);
    }
    __syncthreads();
    if (d.flags & KAN_DELTA_UNIT) {
        unit_factors<DKP>(K, row + kNk * C);
        unit_factors<DKP>(Q, row + kNq * C);
        __syncthreads();
        scale_rows<DKP>(K, row + kNk * C);
        scale_rows<DKP>(Q, row + kNq * C);
        __syncthreads();
    }
    char* const mine = ws;
    const int64_t ch = bh * p.chunks + n;
    float* out_row = reinterpret_cast<float*>(mine + p.off_rows) + ch * kFields * C;
    for (int i = tid; i < kFields * C; i += NT) out_row[i] = i < (kTo + 1) * C ? row[i] : 0.0f;
    float* out_P = reinterpret_cast<float*>(mine + p.off_P) + ch * C * C;
    float* out_Pt = reinterpret_cast<float*>(mine + p.off_Pt) + ch * C * C;
    // this wave's 16 rows of A and P
    for (int jt = 0; jt < 4; ++jt) {
        f32x4 kk = zero4(), qk = zero4();
        if (jt <= wave) {
#pragma unroll
            for (int s = 0; s < DKP / 16; ++s) {
                const f32x4 kb = ld4(K + (16 * jt + r) * (DKP + 4) + 16 * s + 4 * gq);
                mma(kk, ld4(K + (16 * wave + r) * (DKP + 4) + 16 * s + 4 * gq), kb);
                mma(qk, ld4(Q + (16 * wave + r) * (DKP + 4) + 16 * s + 4 * gq), kb);
            }
        }
        const int j = 16 * jt + r;
        f32x4 P;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int i = 16 * wave + 4 * gq + x;
            const float D = j <= i ? decay(row, i, j) : 0.0f;
            A[i * LC + j] = j < i ? kk[x] * D : 0.0f;
            P[x] = j <= i ? d.scale * (qk[x] * D) : 0.0f;
            out_P[i * C + j] = P[x];
        }
        if (BWD) st4(out_Pt + j * C + 16 * wave + 4 * gq, P);
    }
    __syncthreads();
    const float* beta = row + kBeta * C;
    // G = A - A diag(beta) G: the diagonal blocks of 16, a wave each, column r to a lane ...
    {
        float hv[16];                                  // beta_k G[k][r]
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float* Ai = A + (16 * wave + i) * LC + 16 * wave;
            float v = Ai[r];
#pragma unroll
            for (int k = 0; k < i; ++k) v = __builtin_fmaf(-Ai[k], hv[k], v);
            hv[i] = v * beta[16 * wave + i];
            if (gq == 0) G[(16 * wave + i) * LC + 16 * wave + r] = v;
        }
        for (int jt = wave + 1; jt < 4; ++jt)
#pragma unroll
            for (int x = 0; x < 4; ++x) G[(16 * wave + 4 * gq + x) * LC + 16 * jt + r] = 0.0f;
    }
    __syncthreads();
    // ... and the blocks below it, a row of blocks after the other:
    // R = A_ij - sum over k of A_ik diag(beta) G_kj,  G_ij = R - G_ii diag(beta) R
    for (int it = 1; it < 4; ++it) {
        f32x4 R = zero4();
        const int j = 16 * wave + r;
        if (wave < it) {
            for (int kt = wave; kt < it; ++kt) {
                f32x4 gb;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int k = 16 * kt + 4 * gq + x;
                    gb[x] = -beta[k] * G[k * LC + j];
                }
                mma(R, ld4(A + (16 * it + r) * LC + 16 * kt + 4 * gq), gb);
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int i = 16 * it + 4 * gq + x;
                R[x] += A[i * LC + j];
                G[i * LC + j] = R[x];
            }
        }
        __syncthreads();
        if (wave < it) {
            f32x4 gb;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int k = 16 * it + 4 * gq + x;
                gb[x] = -beta[k] * G[k * LC + j];
            }
            mma(R, ld4(G + (16 * it + r) * LC + 16 * it + 4 * gq), gb);
        }
        __syncthreads();
        if (wave < it) {
#pragma unroll
            for (int x = 0; x < 4; ++x) G[(16 * it + 4 * gq + x) * LC + j] = R[x];
        }
        __syncthreads();
    }
    float* out_G = reinterpret_cast<float*>(mine + p.off_G) + ch * C * C;
    float* out_Gt = reinterpret_cast<float*>(mine + p.off_Gt) + ch * C * C;
    for (int e = tid; e < C * C / 4; e += NT) {
        const int i = e >> 4, j = 4 * (e & 15);
        st4(out_G + i * C + j, ld4(G + i * LC + j));
        if (BWD) {
            f32x4 v;
#pragma unroll
            for (int x = 0; x < 4; ++x) v[x] = G[(j + x) * LC + i];
            st4(out_Gt + i * C + j, v);
        }
    }
}

// ---- along a sequence -------------------------------------------------------------

// Columns n0 .. n0 + 31 of the state of head h of sequence b.  A wave has rows 16
// wave .. of what has a chunk's rows, and tiles of 16 x 16 of the state.  BWD: keeps
// the chunks' first states and w for the backward pass and writes no rows.
template <typename TS, int DKP, bool BWD>
__global__ void __launch_bounds__(NT) delta_scan_kernel(kan_delta_desc_t d, DeltaPlan p, DeltaArgs a, char* ws) {
    extern __shared__ float lds[];
    constexpr int LK = DKP + 4;
    constexpr int TILES = DKP / 16 * (NV / 16) / 4;    // of the state, for each wave
    float* K = lds;                                    // [64][LK]
    float* St = K + C * LK;                            // [32][LK]: S transposed
    float* Et = St + NV * LK;                          // [32][LC]: beta e
    float* Ut = Et + NV * LC;                          // [32][LC]: u
    float* row = Ut + NV * LC;                         // [8][64]
    const int tiles = p.dvp / NV;
    const int64_t bh = blockIdx.x / (unsigned)tiles, b = bh / d.Hv, h = bh % d.Hv, hk = h / (d.Hv / d.Hk);
    const int n0 = (int)(blockIdx.x % (unsigned)tiles) * NV;
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, r = lane & 15, gq = lane >> 4;
    const int Dk = (int)d.Dk, Dv = (int)d.Dv, len = length_of(a, b, d.T), chunks = (len + C - 1) / C;
    // tile x of this wave: rows 16 dt of S, columns 16 nt
    auto nt_of = [&](int x) { return (wave + 4 * x) & 1; };
    auto dt_of = [&](int x) { return (wave + 4 * x) >> 1; };
    f32x4 S[TILES];
#pragma unroll
    for (int x = 0; x < TILES; ++x) {
        const int nn = n0 + 16 * nt_of(x) + r;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int dd = 16 * dt_of(x) + 4 * gq + j;
            S[x][j] = a.h0 && dd < Dk && nn < Dv ? a.h0[(bh * Dk + dd) * Dv + nn] : 0.0f;
        }
        st4(St + (16 * nt_of(x) + r) * LK + 16 * dt_of(x) + 4 * gq, S[x]);
    }
    for (int n = 0; n < chunks; ++n) {
        const int64_t ch = bh * p.chunks + n, t0 = (int64_t)n * C;
        const int rows = len - n * C;
        const float* in_row = reinterpret_cast<const float*>(ws + p.off_rows) + ch * kFields * C;
        const float* in_G = reinterpret_cast<const float*>(ws + p.off_G) + ch * C * C;
        const float* in_P = reinterpret_cast<const float*>(ws + p.off_P) + ch * C * C;
        for (int i = tid; i < kFields * C; i += NT) row[i] = in_row[i];
        fill_rows<TS, DKP>(K, static_cast<const TS*>(a.k) + at_row(d.k, b, t0, hk), d.k.row, rows, Dk);
        f32x4 v[2];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = 16 * wave + 4 * gq + j, nn = n0 + 16 * nt + r;
                v[nt][j] = i < rows && nn < Dv ? load_f(static_cast<const TS*>(a.v) + at_row(d.v, b, t0 + i, h), nn)
                                              : 0.0f;
            }
        __syncthreads();
        scale_rows<DKP>(K, row + kNk * C);
        __syncthreads();
        f32x4 ks[2] = {zero4(), zero4()}, qs[2] = {zero4(), zero4()};
        const int iq = 16 * wave + r;
        const TS* q = static_cast<const TS*>(a.q) + at_row(d.q, b, t0 + (iq < rows ? iq : 0), hk);
#pragma unroll
        for (int s = 0; s < DKP / 16; ++s) {
            const int at = 16 * s + 4 * gq;
            const f32x4 ka = ld4(K + iq * LK + at);
            f32x4 qa = zero4();
            if (!BWD && iq < rows) qa = row4<TS>(q, at, Dk);
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
                const f32x4 sb = ld4(St + (16 * nt + r) * LK + at);
                mma(ks[nt], ka, sb);
                if (!BWD) mma(qs[nt], qa, sb);
            }
        }
        if (BWD) {
            float* out = reinterpret_cast<float*>(ws + p.off_S) + ch * DKP * p.dvp;
#pragma unroll
            for (int x = 0; x < TILES; ++x)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    out[(16 * dt_of(x) + 4 * gq + j) * p.dvp + n0 + 16 * nt_of(x) + r] = S[x][j];
        }
        const f32x4 from = ld4(row + kFrom * C + 16 * wave + 4 * gq), beta = ld4(row + kBeta * C + 16 * wave + 4 * gq);
        f32x4 w[2];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
            w[nt] = v[nt] - from * ks[nt];
            st4(Et + (16 * nt + r) * LC + 16 * wave + 4 * gq, beta * w[nt]);
        }
        __syncthreads();
        f32x4 ge[2] = {zero4(), zero4()};
        for (int s = 0; s <= wave; ++s) {
            const f32x4 ga = ld4(in_G + iq * C + 16 * s + 4 * gq);
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) mma(ge[nt], ga, ld4(Et + (16 * nt + r) * LC + 16 * s + 4 * gq));
        }
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
            w[nt] = w[nt] - ge[nt];
            st4(Ut + (16 * nt + r) * LC + 16 * wave + 4 * gq, beta * w[nt]);
            if (BWD) {
                float* out = reinterpret_cast<float*>(ws + p.off_w) + ch * C * p.dvp + n0 + 16 * nt + r;
#pragma unroll
                for (int j = 0; j < 4; ++j) out[(16 * wave + 4 * gq + j) * p.dvp] = w[nt][j];
            }
        }
        __syncthreads();
        if (!BWD) {
            f32x4 o[2] = {zero4(), zero4()};
            for (int s = 0; s <= wave; ++s) {
                const f32x4 pa = ld4(in_P + iq * C + 16 * s + 4 * gq);
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) mma(o[nt], pa, ld4(Ut + (16 * nt + r) * LC + 16 * s + 4 * gq));
            }
            const f32x4 nq = ld4(row + kNq * C + 16 * wave + 4 * gq);
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int i = 16 * wave + 4 * gq + j, nn = n0 + 16 * nt + r;
                    if (i < rows && nn < Dv)
                        put(static_cast<TS*>(a.y) + ((b * d.T + t0 + i) * d.Hv + h) * Dv + nn,
                            o[nt][j] + d.scale * nq[j] * from[j] * qs[nt][j]);
                }
        }
        const float whole = row[kFrom * C + C - 1];
#pragma unroll
        for (int x = 0; x < TILES; ++x) {
            f32x4 add = zero4();
#pragma unroll
            for (int s = 0; s < C / 16; ++s) {
                f32x4 ka;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int i = 16 * s + 4 * gq + j;
                    ka[j] = K[i * LK + 16 * dt_of(x) + r] * row[kTo * C + i];
                }
                mma(add, ka, ld4(Ut + (16 * nt_of(x) + r) * LC + 16 * s + 4 * gq));
            }
            S[x] = whole * S[x] + add;
            st4(St + (16 * nt_of(x) + r) * LK + 16 * dt_of(x) + 4 * gq, S[x]);
        }
        __syncthreads();
    }
    if (BWD) return;
    for (int64_t e = tid; e < (d.T - len) * NV; e += NT) {
        const int64_t t = len + e / NV;
        const int nn = n0 + (int)(e % NV);
        if (nn < Dv) put(static_cast<TS*>(a.y) + ((b * d.T + t) * d.Hv + h) * Dv + nn, 0.0f);
    }
    if (!a.hT) return;
#pragma unroll
    for (int x = 0; x < TILES; ++x) {
        const int nn = n0 + 16 * nt_of(x) + r;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int dd = 16 * dt_of(x) + 4 * gq + j;
            if (dd < Dk && nn < Dv) a.hT[(bh * Dk + dd) * Dv + nn] = S[x][j];
        }
    }
}

// Backwards along a sequence: r, dv and the gradients of the chunks' last states.
template <typename TS, int DKP>
__global__ void __launch_bounds__(NT) delta_back_kernel(kan_delta_desc_t d, DeltaPlan p, DeltaArgs a, char* ws) {
    extern __shared__ float lds[];
    constexpr int LK = DKP + 4;
    constexpr int TILES = DKP / 16 * (NV / 16) / 4;
    float* K = lds;                                    // [64][LK]
    float* Q = K + C * LK;                             // [64][LK]
    float* St = Q + C * LK;                            // [32][LK]: dS transposed
    float* Yt = St + NV * LK;                          // [32][LC]: dY
    float* Ut = Yt + NV * LC;                          // [32][LC]: beta du, then dv
    float* row = Ut + NV * LC;                         // [8][64]
    const int tiles = p.dvp / NV;
    const int64_t bh = blockIdx.x / (unsigned)tiles, b = bh / d.Hv, h = bh % d.Hv, hk = h / (d.Hv / d.Hk);
    const int n0 = (int)(blockIdx.x % (unsigned)tiles) * NV;
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, r = lane & 15, gq = lane >> 4;
    const int Dk = (int)d.Dk, Dv = (int)d.Dv, len = length_of(a, b, d.T), chunks = (len + C - 1) / C;
    auto nt_of = [&](int x) { return (wave + 4 * x) & 1; };
    auto dt_of = [&](int x) { return (wave + 4 * x) >> 1; };
    for (int64_t e = tid; e < (d.T - len) * NV; e += NT) {
        const int64_t t = len + e / NV;
        const int nn = n0 + (int)(e % NV);
        if (nn < Dv) put(static_cast<TS*>(a.dv) + at_row(d.dv, b, t, h) + nn, 0.0f);
    }
    f32x4 S[TILES];
#pragma unroll
    for (int x = 0; x < TILES; ++x) {
        const int nn = n0 + 16 * nt_of(x) + r;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int dd = 16 * dt_of(x) + 4 * gq + j;
            S[x][j] = a.dhT && dd < Dk && nn < Dv ? a.dhT[(bh * Dk + dd) * Dv + nn] : 0.0f;
        }
        st4(St + (16 * nt_of(x) + r) * LK + 16 * dt_of(x) + 4 * gq, S[x]);
    }
    for (int n = chunks - 1; n >= 0; --n) {
        const int64_t ch = bh * p.chunks + n, t0 = (int64_t)n * C;
        const int rows = len - n * C;
        const float* in_row = reinterpret_cast<const float*>(ws + p.off_rows) + ch * kFields * C;
        const float* in_Gt = reinterpret_cast<const float*>(ws + p.off_Gt) + ch * C * C;
        const float* in_Pt = reinterpret_cast<const float*>(ws + p.off_Pt) + ch * C * C;
        for (int i = tid; i < kFields * C; i += NT) row[i] = in_row[i];
        fill_rows<TS, DKP>(K, static_cast<const TS*>(a.k) + at_row(d.k, b, t0, hk), d.k.row, rows, Dk);
        fill_rows<TS, DKP>(Q, static_cast<const TS*>(a.q) + at_row(d.q, b, t0, hk), d.q.row, rows, Dk);
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
            f32x4 y;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = 16 * wave + 4 * gq + j, nn = n0 + 16 * nt + r;
                y[j] = i < rows && nn < Dv
                           ? load_f(static_cast<const TS*>(a.dy) + ((b * d.T + t0 + i) * d.Hv + h) * Dv, nn)
                           : 0.0f;
            }
            st4(Yt + (16 * nt + r) * LC + 16 * wave + 4 * gq, y);
        }
        float* out_S = reinterpret_cast<float*>(ws + p.off_dS) + ch * DKP * p.dvp;
#pragma unroll
        for (int x = 0; x < TILES; ++x)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                out_S[(16 * dt_of(x) + 4 * gq + j) * p.dvp + n0 + 16 * nt_of(x) + r] = S[x][j];
        __syncthreads();
        scale_rows<DKP>(K, row + kNk * C);
        scale_rows<DKP>(Q, row + kNq * C);
        __syncthreads();
        const int iq = 16 * wave + r;
        f32x4 kd[2] = {zero4(), zero4()}, py[2] = {zero4(), zero4()};
#pragma unroll
        for (int s = 0; s < DKP / 16; ++s) {
            const f32x4 ka = ld4(K + iq * LK + 16 * s + 4 * gq);
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) mma(kd[nt], ka, ld4(St + (16 * nt + r) * LK + 16 * s + 4 * gq));
        }
        for (int s = wave; s < 4; ++s) {
            const f32x4 pa = ld4(in_Pt + iq * C + 16 * s + 4 * gq);
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) mma(py[nt], pa, ld4(Yt + (16 * nt + r) * LC + 16 * s + 4 * gq));
        }
        const f32x4 to = ld4(row + kTo * C + 16 * wave + 4 * gq), beta = ld4(row + kBeta * C + 16 * wave + 4 * gq);
        const f32x4 from = ld4(row + kFrom * C + 16 * wave + 4 * gq);
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
            py[nt] = py[nt] + to * kd[nt];             // du
            st4(Ut + (16 * nt + r) * LC + 16 * wave + 4 * gq, beta * py[nt]);
        }
        __syncthreads();
        f32x4 gu[2] = {zero4(), zero4()};
        for (int s = wave; s < 4; ++s) {
            const f32x4 ga = ld4(in_Gt + iq * C + 16 * s + 4 * gq);
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) mma(gu[nt], ga, ld4(Ut + (16 * nt + r) * LC + 16 * s + 4 * gq));
        }
        __syncthreads();
        float* out_r = reinterpret_cast<float*>(ws + p.off_r) + ch * C * p.dvp + n0;
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
            const f32x4 rr = py[nt] - gu[nt], dv = beta * rr;
            // rows of dS0: exp(c) (scale q dY - k dv), dY and dv with their factor
            st4(Ut + (16 * nt + r) * LC + 16 * wave + 4 * gq, from * dv);
            float* y = Yt + (16 * nt + r) * LC + 16 * wave + 4 * gq;
            st4(y, ld4(y) * from * d.scale);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = 16 * wave + 4 * gq + j, nn = n0 + 16 * nt + r;
                out_r[i * p.dvp + 16 * nt + r] = rr[j];
                if (i < rows && nn < Dv) put(static_cast<TS*>(a.dv) + at_row(d.dv, b, t0 + i, h) + nn, dv[j]);
            }
        }
        __syncthreads();
        const float whole = row[kFrom * C + C - 1];
#pragma unroll
        for (int x = 0; x < TILES; ++x) {
            f32x4 add = zero4(), sub = zero4();
#pragma unroll
            for (int s = 0; s < C / 16; ++s) {
                f32x4 ka, qa;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int i = 16 * s + 4 * gq + j;
                    ka[j] = K[i * LK + 16 * dt_of(x) + r];
                    qa[j] = Q[i * LK + 16 * dt_of(x) + r];
                }
                mma(add, qa, ld4(Yt + (16 * nt_of(x) + r) * LC + 16 * s + 4 * gq));
                mma(sub, ka, ld4(Ut + (16 * nt_of(x) + r) * LC + 16 * s + 4 * gq));
            }
            S[x] = whole * S[x] + (add - sub);
            st4(St + (16 * nt_of(x) + r) * LK + 16 * dt_of(x) + 4 * gq, S[x]);
        }
        __syncthreads();
    }
    if (!a.dh0) return;
#pragma unroll
    for (int x = 0; x < TILES; ++x) {
        const int nn = n0 + 16 * nt_of(x) + r;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int dd = 16 * dt_of(x) + 4 * gq + j;
            if (dd < Dk && nn < Dv) a.dh0[(bh * Dk + dd) * Dv + nn] = S[x][j];
        }
    }
}

// ---- gradients of a chunk's rows -----------------------------------------------------

// 16 x 16 values of a wave, summed over each row's 16 lanes: all of them get it.
__device__ __forceinline__ f32x4 row_sums(f32x4 v) {
#pragma unroll
    for (int o = 1; o < 16; o <<= 1)
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] += __shfl_xor(v[j], o, 64);
    return v;
}

template <typename TS, int DKP>
__global__ void __launch_bounds__(NT) delta_grad_kernel(kan_delta_desc_t d, DeltaPlan p, DeltaArgs a, char* ws) {
    extern __shared__ float lds[];
    constexpr int LK = DKP + 4, DT = DKP / 16;
    float* K = lds;                                    // [64][LK]
    float* Q = K + C * LK;
    float* PD = Q + C * LK;                            // [64][LC]: scale dP D
    float* XD = PD + C * LC;                           // X D
    float* E = XD + C * LC;                            // dP P - X A, and its sums along rows
    float* row = E + C * LC;                           // [8][64]
    float* xs = row + kFields * C;                     // [64] parts of rows that come from S0
    float* zs = xs + C;                                // [64] parts of rows that reach dS1
    float* part = zs + C;                              // [4] of <dS1, S0>
    const int64_t n = blockIdx.x % (unsigned)p.chunks, bh = blockIdx.x / (unsigned)p.chunks;
    const int64_t b = bh / d.Hv, h = bh % d.Hv, share = d.Hv / d.Hk, hk = h / share;
    const int64_t t0 = n * C, ch = bh * p.chunks + n;
    const int Dk = (int)d.Dk, Dv = (int)d.Dv;
    const int rows = length_of(a, b, d.T) - (int)t0;
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, r = lane & 15, gq = lane >> 4;
    const int inside = (int)(d.T - t0 < C ? d.T - t0 : C);   // rows of the chunk that the arrays have
    TS* const dq = static_cast<TS*>(a.dq) + at_row(d.dq, b, t0, hk);
    TS* const dk = static_cast<TS*>(a.dk) + at_row(d.dk, b, t0, hk);
    float* const part_q = reinterpret_cast<float*>(ws + p.off_dq) + ((b * d.T + t0) * d.Hv + h) * Dk;
    float* const part_k = reinterpret_cast<float*>(ws + p.off_dk) + ((b * d.T + t0) * d.Hv + h) * Dk;
    if (rows <= 0) {                                   // uniform
        if (tid < inside) {
            a.dg[(b * d.T + t0 + tid) * d.Hv + h] = 0.0f;
            a.dbeta[(b * d.T + t0 + tid) * d.Hv + h] = 0.0f;
        }
        if (share == 1)
            for (int e = tid; e < inside * Dk; e += NT) {
                put(dq + e / Dk * d.dq.row + e % Dk, 0.0f);
                put(dk + e / Dk * d.dk.row + e % Dk, 0.0f);
            }
        return;
    }
    const float* in_row = reinterpret_cast<const float*>(ws + p.off_rows) + ch * kFields * C;
    for (int i = tid; i < kFields * C; i += NT) row[i] = in_row[i];
    fill_rows<TS, DKP>(K, static_cast<const TS*>(a.k) + at_row(d.k, b, t0, hk), d.k.row, rows, Dk);
    fill_rows<TS, DKP>(Q, static_cast<const TS*>(a.q) + at_row(d.q, b, t0, hk), d.q.row, rows, Dk);
    __syncthreads();
    scale_rows<DKP>(K, row + kNk * C);
    scale_rows<DKP>(Q, row + kNq * C);
    __syncthreads();
    const float* S0 = reinterpret_cast<const float*>(ws + p.off_S) + ch * DKP * p.dvp;
    const float* dS = reinterpret_cast<const float*>(ws + p.off_dS) + ch * DKP * p.dvp;
    const float* in_w = reinterpret_cast<const float*>(ws + p.off_w) + ch * C * p.dvp;
    const float* in_r = reinterpret_cast<const float*>(ws + p.off_r) + ch * C * p.dvp;
    const int im = 16 * wave + r;                      // this lane's row of A operands
    const float beta_m = row[kBeta * C + im];
    const TS* dy = static_cast<const TS*>(a.dy) + ((b * d.T + t0 + (im < rows ? im : 0)) * d.Hv + h) * Dv;
    f32x4 ys[DT], vs[DT], us[DT], dP[4], X[4];
#pragma unroll
    for (int x = 0; x < DT; ++x) ys[x] = vs[x] = us[x] = zero4();
#pragma unroll
    for (int x = 0; x < 4; ++x) dP[x] = X[x] = zero4();
    float rw = 0.0f, ss = 0.0f;
    for (int s = 0; s < p.dvp / 16; ++s) {
        const int at = 16 * s + 4 * gq;
        const f32x4 ya = im < rows ? row4<TS>(dy, at, Dv) : zero4();
        const f32x4 wa = ld4(in_w + im * p.dvp + at), ra = ld4(in_r + im * p.dvp + at);
        const f32x4 ua = beta_m * wa, va = beta_m * ra;
#pragma unroll
        for (int j = 0; j < 4; ++j) rw = __builtin_fmaf(wa[j], ra[j], rw);
#pragma unroll
        for (int x = 0; x < DT; ++x) {
            const f32x4 sb = ld4(S0 + (16 * x + r) * p.dvp + at), db = ld4(dS + (16 * x + r) * p.dvp + at);
            mma(ys[x], ya, sb);
            mma(vs[x], va, sb);
            mma(us[x], ua, db);
            if ((x & 3) == wave)
#pragma unroll
                for (int j = 0; j < 4; ++j) ss = __builtin_fmaf(sb[j], db[j], ss);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            if (x > wave) break;
            const f32x4 ub = row[kBeta * C + 16 * x + r] * ld4(in_w + (16 * x + r) * p.dvp + at);
            mma(dP[x], ya, ub);
            mma(X[x], va, ub);
        }
    }
    rw += __shfl_xor(rw, 16, 64);
    rw += __shfl_xor(rw, 32, 64);
    if (gq == 0 && im < inside) a.dbeta[(b * d.T + t0 + im) * d.Hv + h] = im < rows ? rw : 0.0f;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) ss += __shfl_xor(ss, o, 64);
    if (lane == 0) part[wave] = ss;
    // the states' parts, with their factors
    const f32x4 from = ld4(row + kFrom * C + 16 * wave + 4 * gq), to = ld4(row + kTo * C + 16 * wave + 4 * gq);
    f32x4 xr = zero4(), zr = zero4();
#pragma unroll
    for (int x = 0; x < DT; ++x) {
        ys[x] = d.scale * (from * ys[x]);
        vs[x] = from * vs[x];
        us[x] = to * us[x];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int at = (16 * wave + 4 * gq + j) * LK + 16 * x + r;
            xr[j] += Q[at] * ys[x][j] - K[at] * vs[x][j];
            zr[j] += K[at] * us[x][j];
        }
        us[x] = us[x] - vs[x];                         // dk so far; ys: dq so far
    }
    xr = row_sums(xr);
    zr = row_sums(zr);
    if (r == 0) {
        st4(xs + 16 * wave + 4 * gq, xr);
        st4(zs + 16 * wave + 4 * gq, zr);
    }
    // pairs of rows
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        f32x4 qk = zero4(), kk = zero4();
        if (x <= wave) {
#pragma unroll
            for (int s = 0; s < DT; ++s) {
                const f32x4 kb = ld4(K + (16 * x + r) * LK + 16 * s + 4 * gq);
                mma(qk, ld4(Q + im * LK + 16 * s + 4 * gq), kb);
                mma(kk, ld4(K + im * LK + 16 * s + 4 * gq), kb);
            }
        }
        const int j = 16 * x + r;
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            const int i = 16 * wave + 4 * gq + y;
            const float D = j <= i ? decay(row, i, j) : 0.0f;
            const float pd = j <= i ? d.scale * (dP[x][y] * D) : 0.0f, xd = j < i ? X[x][y] * D : 0.0f;
            PD[i * LC + j] = pd;
            XD[i * LC + j] = xd;
            E[i * LC + j] = j < i ? pd * qk[y] - xd * kk[y] : 0.0f;
        }
    }
    __syncthreads();
    // products of the pairs with the rows; rows of K and Q as columns
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        f32x4 pt, xt;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            pt[j] = PD[(16 * s + 4 * gq + j) * LC + im];
            xt[j] = XD[(16 * s + 4 * gq + j) * LC + im];
        }
        const f32x4 pa = ld4(PD + im * LC + 16 * s + 4 * gq), xa = ld4(XD + im * LC + 16 * s + 4 * gq) + xt;
#pragma unroll
        for (int x = 0; x < DT; ++x) {
            f32x4 kb, qb;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                kb[j] = K[(16 * s + 4 * gq + j) * LK + 16 * x + r];
                qb[j] = Q[(16 * s + 4 * gq + j) * LK + 16 * x + r];
            }
            if (s <= wave) mma(ys[x], pa, kb);
            if (s >= wave) mma(us[x], pt, qb);
            mma(us[x], -xa, kb);
        }
    }
    // dg: sums of E along rows (wave 0, a row to a lane), then down the columns
    if (wave == 0) {
        float sum = 0.0f;
        for (int j = 0; j < C; ++j) {
            const float e = E[lane * LC + j];
            E[lane * LC + j] = sum;                    // over the columns before j
            sum += e;
        }
    }
    __syncthreads();
    if (wave == 0) {
        float dg = 0.0f;
        for (int i = C - 1; i >= lane; --i) dg += E[i * LC + lane] + xs[i];
        for (int j = 0; j < lane; ++j) dg += zs[j];
        dg += row[kFrom * C + C - 1] * (part[0] + part[1] + part[2] + part[3]);
        if (lane < inside) a.dg[(b * d.T + t0 + lane) * d.Hv + h] = lane < rows ? dg : 0.0f;
    }
    if (share > 1) {
#pragma unroll
        for (int x = 0; x < DT; ++x)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = 16 * wave + 4 * gq + j, dd = 16 * x + r;
                if (i < rows && dd < Dk) {
                    part_q[(int64_t)i * d.Hv * Dk + dd] = ys[x][j];
                    part_k[(int64_t)i * d.Hv * Dk + dd] = us[x][j];
                }
            }
        return;
    }
    if (d.flags & KAN_DELTA_UNIT) {                    // through x / sqrt(x.x + eps), x here already divided
        f32x4 qd = zero4(), kd = zero4();
#pragma unroll
        for (int x = 0; x < DT; ++x)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int at = (16 * wave + 4 * gq + j) * LK + 16 * x + r;
                qd[j] += Q[at] * ys[x][j];
                kd[j] += K[at] * us[x][j];
            }
        qd = row_sums(qd);
        kd = row_sums(kd);
        const f32x4 nq = ld4(row + kNq * C + 16 * wave + 4 * gq), nk = ld4(row + kNk * C + 16 * wave + 4 * gq);
#pragma unroll
        for (int x = 0; x < DT; ++x)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int at = (16 * wave + 4 * gq + j) * LK + 16 * x + r;
                ys[x][j] = nq[j] * (ys[x][j] - Q[at] * qd[j]);
                us[x][j] = nk[j] * (us[x][j] - K[at] * kd[j]);
            }
    }
#pragma unroll
    for (int x = 0; x < DT; ++x)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = 16 * wave + 4 * gq + j, dd = 16 * x + r;
            if (i < inside && dd < Dk) {
                put(dq + i * d.dq.row + dd, i < rows ? ys[x][j] : 0.0f);
                put(dk + i * d.dk.row + dd, i < rows ? us[x][j] : 0.0f);
            }
        }
}

// Heads that share a key: their gradients summed in order, a wave to a row of q
// and k each.
template <typename TS>
__global__ void __launch_bounds__(NT) delta_heads_kernel(kan_delta_desc_t d, DeltaPlan p, DeltaArgs a,
                                                         const char* ws) {
    const int64_t at = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * (NT / 64) + (threadIdx.x >> 6);
    if (at >= d.B * d.T * d.Hk) return;
    const int lane = threadIdx.x & 63, Dk = (int)d.Dk;
    const int64_t b = at / (d.T * d.Hk), t = at / d.Hk % d.T, hk = at % d.Hk, share = d.Hv / d.Hk;
    const bool inside = t < length_of(a, b, d.T);
#pragma unroll
    for (int z = 0; z < 2; ++z) {
        const kan_heads_t& si = z ? d.k : d.q;
        const kan_heads_t& so = z ? d.dk : d.dq;
        const TS* x = static_cast<const TS*>(z ? a.k : a.q) + at_row(si, b, t, hk);
        TS* out = static_cast<TS*>(z ? a.dk : a.dq) + at_row(so, b, t, hk);
        const float* part = reinterpret_cast<const float*>(ws + (z ? p.off_dk : p.off_dq)) +
                            ((b * d.T + t) * d.Hv + hk * share) * Dk;
        float v[2] = {0.0f, 0.0f}, in[2] = {0.0f, 0.0f}, dot = 0.0f, sq = 0.0f;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const int dd = lane + 64 * m;
            if (!inside || dd >= Dk) continue;
            for (int64_t s = 0; s < share; ++s) v[m] += part[s * Dk + dd];
            in[m] = load_f(x, dd);
            dot += in[m] * v[m], sq += in[m] * in[m];
        }
        if (d.flags & KAN_DELTA_UNIT) {
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) dot += __shfl_xor(dot, o, 64), sq += __shfl_xor(sq, o, 64);
            const float f = 1.0f / sqrtf(sq + kUnitEps);
#pragma unroll
            for (int m = 0; m < 2; ++m) v[m] = f * (v[m] - in[m] * f * (f * dot));
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const int dd = lane + 64 * m;
            if (dd < Dk) put(out + dd, inside ? v[m] : 0.0f);
        }
    }
}

// ---- one row -----------------------------------------------------------------------

// Columns 64 blk .. of head h's state of sequence b: 16 lanes of four columns, 16
// rows of threads along Dk, eight rows of the state to a thread.
template <typename TS>
__global__ void __launch_bounds__(NT) delta_step_kernel(kan_delta_desc_t d, int64_t pool, DeltaArgs a, float* state,
                                                        const int32_t* slots, int tiles) {
    __shared__ float ks[kDeltaMaxDk], qs[kDeltaMaxDk], red[2][16][68], factor[2];
    const int64_t bh = blockIdx.x / (unsigned)tiles, b = bh / d.Hv, h = bh % d.Hv, hk = h / (d.Hv / d.Hk);
    const int n0 = (int)(blockIdx.x % (unsigned)tiles) * 64, tid = threadIdx.x;
    const int Dk = (int)d.Dk, Dv = (int)d.Dv;
    const int64_t slot = slots ? slots[b] : b;
    TS* y = static_cast<TS*>(a.y) + (b * d.Hv + h) * Dv;
    if (slot < 0 || slot >= pool) {
        if (tid < 64 && n0 + tid < Dv) put(y + n0 + tid, 0.0f);
        return;
    }
    if (tid < 128) {
        const int lane = tid & 63;
        const TS* x = tid < 64 ? static_cast<const TS*>(a.k) + b * d.k.seq + hk * d.k.head
                               : static_cast<const TS*>(a.q) + b * d.q.seq + hk * d.q.head;
        const float x0 = lane < Dk ? load_f(x, lane) : 0.0f, x1 = lane + 64 < Dk ? load_f(x, lane + 64) : 0.0f;
        float* to = tid < 64 ? ks : qs;
        float f = 1.0f;
        if (d.flags & KAN_DELTA_UNIT) {
            float n = x0 * x0 + x1 * x1;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) n += __shfl_xor(n, o, 64);
            f = 1.0f / sqrtf(n + kUnitEps);
        }
        to[lane] = x0 * f;
        to[lane + 64] = x1 * f;
    }
    float g = a.g[b * d.Hv + h];
    const float alpha = expf(g < -128.0f ? -128.0f : g), beta = a.beta[b * d.Hv + h];
    const int c = tid & 15, rt = tid >> 4, nn = n0 + 4 * c;
    float* S = state + (slot * d.Hv + h) * Dk * Dv;
    f32x4 s[8];
#pragma unroll
    for (int m = 0; m < 8; ++m) {
        const int dd = rt + 16 * m;
        s[m] = dd < Dk ? row4<float>(S + (int64_t)dd * Dv, nn, Dv) * alpha : zero4();
    }
    __syncthreads();
    f32x4 w = zero4();
#pragma unroll
    for (int m = 0; m < 8; ++m) w += ks[rt + 16 * m] * s[m];
    st4(&red[0][rt][4 * c], w);
    const TS* v = static_cast<const TS*>(a.v) + b * d.v.seq + h * d.v.head;
    f32x4 u = row4<TS>(v, nn, Dv);
    __syncthreads();
    w = zero4();
#pragma unroll
    for (int m = 0; m < 16; ++m) w += ld4(&red[0][m][4 * c]);
    u = beta * (u - w);
    f32x4 o = zero4();
#pragma unroll
    for (int m = 0; m < 8; ++m) {
        const int dd = rt + 16 * m;
        s[m] += ks[dd] * u;
        o += qs[dd] * s[m];
        if (dd < Dk) {
            float* to = S + (int64_t)dd * Dv + nn;
            if (nn + 4 <= Dv) {
                const float t[4] = {s[m][0], s[m][1], s[m][2], s[m][3]};
                store_vec<4>(to, t);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (nn + j < Dv) to[j] = s[m][j];
            }
        }
    }
    st4(&red[1][rt][4 * c], o);
    __syncthreads();
    if (tid < 64 && n0 + tid < Dv) {
        float sum = 0.0f;
#pragma unroll
        for (int m = 0; m < 16; ++m) sum += red[1][m][tid];
        put(y + n0 + tid, d.scale * sum);
    }
}

// ---- launches ----------------------------------------------------------------------

template <typename K>
hipError_t set_lds(K kernel, size_t bytes) {
    return hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize,
                               (int)bytes);
}

template <typename TS, int DKP, bool BWD>
hipError_t prep(const kan_delta_desc_t& d, const DeltaPlan& p, const DeltaArgs& a, char* ws, hipStream_t s) {
    constexpr size_t lds = 4 * (2 * C * (DKP + 4) + 2 * C * LC + kFields * C);
    const hipError_t e = set_lds(delta_prep_kernel<TS, DKP, BWD>, lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((delta_prep_kernel<TS, DKP, BWD>), dim3((unsigned)(p.heads * p.chunks)), dim3(NT), lds, s, d, p,
                       a, ws);
    return hipGetLastError();
}
template <typename TS, int DKP, bool BWD>
hipError_t scan(const kan_delta_desc_t& d, const DeltaPlan& p, const DeltaArgs& a, char* ws, hipStream_t s) {
    constexpr size_t lds = 4 * ((C + NV) * (DKP + 4) + 2 * NV * LC + kFields * C);
    const hipError_t e = set_lds(delta_scan_kernel<TS, DKP, BWD>, lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((delta_scan_kernel<TS, DKP, BWD>), dim3((unsigned)(p.heads * (p.dvp / NV))), dim3(NT), lds, s, d,
                       p, a, ws);
    return hipGetLastError();
}
template <typename TS, int DKP>
hipError_t forward(const kan_delta_desc_t& d, const DeltaPlan& p, const DeltaArgs& a, char* ws, hipStream_t s) {
    if (p.chunks > 0) {
        const hipError_t e = prep<TS, DKP, false>(d, p, a, ws, s);
        if (e != hipSuccess) return e;
    }
    return scan<TS, DKP, false>(d, p, a, ws, s);
}
template <typename TS, int DKP>
hipError_t backward(const kan_delta_desc_t& d, const DeltaPlan& p, const DeltaArgs& a, char* ws, hipStream_t s) {
    hipError_t e;
    if (p.chunks > 0) {
        if ((e = prep<TS, DKP, true>(d, p, a, ws, s)) != hipSuccess) return e;
        if ((e = scan<TS, DKP, true>(d, p, a, ws, s)) != hipSuccess) return e;
    }
    constexpr size_t lds_b = 4 * ((2 * C + NV) * (DKP + 4) + 2 * NV * LC + kFields * C);
    if ((e = set_lds(delta_back_kernel<TS, DKP>, lds_b)) != hipSuccess) return e;
    hipLaunchKernelGGL((delta_back_kernel<TS, DKP>), dim3((unsigned)(p.heads * (p.dvp / NV))), dim3(NT), lds_b, s, d, p,
                       a, ws);
    if ((e = hipGetLastError()) != hipSuccess || p.chunks == 0) return e;
    constexpr size_t lds_g = 4 * (2 * C * (DKP + 4) + 3 * C * LC + kFields * C + 2 * C + 4);
    if ((e = set_lds(delta_grad_kernel<TS, DKP>, lds_g)) != hipSuccess) return e;
    hipLaunchKernelGGL((delta_grad_kernel<TS, DKP>), dim3((unsigned)(p.heads * p.chunks)), dim3(NT), lds_g, s, d, p, a,
                       ws);
    if ((e = hipGetLastError()) != hipSuccess || d.Hv == d.Hk) return e;
    const int64_t blocks = (d.B * d.T * d.Hk + NT / 64 - 1) / (NT / 64), x = std::min<int64_t>(blocks, 1 << 16);
    hipLaunchKernelGGL((delta_heads_kernel<TS>), dim3((unsigned)x, (unsigned)((blocks + x - 1) / x)), dim3(NT), 0, s, d,
                       p, a, (const char*)ws);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_fwd(const kan_delta_desc_t& d, const DeltaPlan& p, const DeltaArgs& a, char* ws,
                            hipStream_t s) {
    if (d.dtype == KAN_F32)
        return p.dkp == 32 ? forward<float, 32>(d, p, a, ws, s)
                           : p.dkp == 64 ? forward<float, 64>(d, p, a, ws, s) : forward<float, 128>(d, p, a, ws, s);
    return p.dkp == 32 ? forward<uint16_t, 32>(d, p, a, ws, s)
                       : p.dkp == 64 ? forward<uint16_t, 64>(d, p, a, ws, s) : forward<uint16_t, 128>(d, p, a, ws, s);
}
hipError_t launch_delta_bwd(const kan_delta_desc_t& d, const DeltaPlan& p, const DeltaArgs& a, char* ws,
                            hipStream_t s) {
    if (d.dtype == KAN_F32)
        return p.dkp == 32 ? backward<float, 32>(d, p, a, ws, s)
                           : p.dkp == 64 ? backward<float, 64>(d, p, a, ws, s) : backward<float, 128>(d, p, a, ws, s);
    return p.dkp == 32 ? backward<uint16_t, 32>(d, p, a, ws, s)
                       : p.dkp == 64 ? backward<uint16_t, 64>(d, p, a, ws, s) : backward<uint16_t, 128>(d, p, a, ws, s);
}
hipError_t launch_delta_step(const kan_delta_desc_t& d, int64_t S, const DeltaArgs& a, float* state,
                             const int32_t* slots, hipStream_t s) {
    const int tiles = (int)((d.Dv + 63) / 64);
    const dim3 grid((unsigned)(d.B * d.Hv * tiles));
    if (d.dtype == KAN_F32)
        hipLaunchKernelGGL(delta_step_kernel<float>, grid, dim3(NT), 0, s, d, S, a, state, slots, tiles);
    else
        hipLaunchKernelGGL(delta_step_kernel<uint16_t>, grid, dim3(NT), 0, s, d, S, a, state, slots, tiles);
    return hipGetLastError();
}

}  // namespace kan
