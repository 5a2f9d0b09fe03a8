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

constexpr int C = kDeltaChunk;
constexpr int LC = C + 4;            // LDS pitch of 64 floats: rows 16 bytes apart modulo the banks
constexpr float kUnitEps = 1e-6f;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// What a chunk's rows have for themselves: [8][64] floats of a chunk-head.
enum RowField {
    kBeta,
    kFk,                             // exp(c) / |k|, |k| where rows are made unit vectors, else 1
    kTk,                             // exp(c_63 - c) / |k|
    kFq,                             // scale exp(c) / |q|
    kNk,                             // 1 / |k|
    kNq,                             // 1 / |q|
    kHi,                             // c log2(e) as the sum of two floats
    kLo,
    kFields
};

__device__ __forceinline__ f32x4 zero4() { return f32x4{0.0f, 0.0f, 0.0f, 0.0f}; }
__device__ __forceinline__ f32x4 ld4(const float* p) { return *reinterpret_cast<const f32x4*>(p); }
__device__ __forceinline__ void st4(float* p, const f32x4& v) { *reinterpret_cast<f32x4*>(p) = v; }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t* p, float v) { *p = f2bf(v); }

// ---- products of matrices ----------------------------------------------------------
//
// v_mfma_f32_16x16x32_bf16: lane l = 16 gq + m has row m of the left operand (or
// column m of the right one) at eight values of the contracted index, and rows 4
// gq .. 4 gq + 3 of column m of the result.  A float is the sum of three bfloat16s,
// a plane each (24 bits); of two operands' planes the products are added whose
// place is within those 24 bits: six for two floats, three where one operand is
// bfloat16 as it stands.  That is 2.7 and 5.3 times as fast as float32's own
// instruction, and as exact.  An answer stored as bfloat16 is a sum of terms that
// may cancel, so that its floats (P, u and the state) have three planes as well; with
// two 8 x 4096 x 16 x 128 bf16 forward takes 424 us and not 460.
//
// The result of one product is an operand of the next without leaving its
// lanes: of 32 values of a contracted index, lane (gq, m) takes 8 gq .. 8 gq + 7,
// and two tiles 2 s, 2 s + 1 of a result have rows 32 s + 8 gq + 4 (tile % 2) + 0 .. 3 in
// the lanes of gq.
__device__ __forceinline__ int row_of(int tile, int m) { return 32 * (tile >> 1) + 8 * (m >> 2) + 4 * (tile & 1) + (m & 3); }

// acc += sum over planes of a b, the small ones first
template <int NA, int NB>
__device__ __forceinline__ void mma(f32x4& acc, const bf16x8 (&a)[NA], const bf16x8 (&b)[NB]) {
    constexpr int N = NA > NB ? NA : NB;
#pragma unroll
    for (int place = N - 1; place >= 0; --place)
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (place - i >= 0 && place - i < NB)
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i], b[place - i], acc, 0, 0, 0);
}

// Eight floats as N planes; every plane takes the rounding of what is left.
template <int N>
__device__ __forceinline__ void split8(f32x4 a, f32x4 b, bf16x8 (&out)[N]) {
    uint32_t w[N][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float x = i < 2 ? a[2 * i] : b[2 * i - 4], y = i < 2 ? a[2 * i + 1] : b[2 * i - 3];
#pragma unroll
        for (int n = 0; n < N; ++n) {
            w[n][i] = pack_bf16(x, y);
            x -= __uint_as_float(w[n][i] << 16);
            y -= __uint_as_float(w[n][i] & 0xffff0000u);
        }
    }
#pragma unroll
    for (int n = 0; n < N; ++n) __builtin_memcpy(&out[n], w[n], 16);
}

// ---- rows in LDS ---------------------------------------------------------------------
//
// 64 rows of W bfloat16s, a plane after the other, in pieces of eight.  A row's
// pieces are permuted so that the 16 rows of a tile, and the four rows by four
// pieces of a transposed read, lie in different banks.
template <int W>
__device__ __forceinline__ int piece_at(int row, int c) {
    constexpr int CH = W / 8;
    return (row * CH + (c ^ ((((row & 3) << 2) | ((row >> 3) & 3)) & (CH - 1)))) * 8;
}
// Planes of pieces 32 s + 8 gq .. of a row: an operand's row, contracted along it.
template <int PL, int W>
__device__ __forceinline__ void row_frag(const uint16_t* lds, int row, int c, bf16x8 (&out)[PL]) {
#pragma unroll
    for (int n = 0; n < PL; ++n) out[n] = *reinterpret_cast<const bf16x8*>(lds + n * C * W + piece_at<W>(row, c));
}
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
// The transposed operand: column `m` of 16, contracted along rows 32 s + 8 gq .. + 7.
// The columns are those of pieces `c` to `c + PIECES - 1`, four a lane: lane 4 a + b of 16
// reads four columns from row a; `c` and `half` are those of lane b.
template <int PL, int W>
__device__ __forceinline__ void col_frag(const uint16_t* lds, int s, int c, int half, bf16x8 (&out)[PL]) {
    const int lane = threadIdx.x & 63, row = 32 * s + 8 * (lane >> 4) + ((lane & 15) >> 2);
#pragma unroll
    for (int n = 0; n < PL; ++n) {
        s16x4 v[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
            v[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lds_s16x4*)(lds + n * C * W + piece_at<W>(row + 4 * h, c) + 4 * half));
        __builtin_memcpy(&out[n], v, 16);
    }
}

// Eight elements of a row on their way from HBM to LDS.
template <typename TS>
struct Piece {
    float v[8];
};
template <>
struct Piece<uint16_t> {
    uint32_t w[4];
};
__device__ __forceinline__ void load_whole(Piece<uint16_t>& p, const uint16_t* from) {
    const Raw<uint16_t, 8> r = load_raw<uint16_t, 8>(from);
#pragma unroll
    for (int i = 0; i < 4; ++i) p.w[i] = r.w[i];
}
__device__ __forceinline__ void load_whole(Piece<float>& p, const float* from) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const Raw<float, 4> r = load_raw<float, 4>(from + 4 * h);
#pragma unroll
        for (int i = 0; i < 4; ++i) p.v[4 * h + i] = raw_value(r, i);
    }
}
__device__ __forceinline__ void load_piece(Piece<uint16_t>& p, const uint16_t* row, int at, int D) {
    if (at + 8 <= D) return load_whole(p, row + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        p.w[i] = at + 2 * i < D ? row[at + 2 * i] : 0u;
        if (at + 2 * i + 1 < D) p.w[i] |= (uint32_t)row[at + 2 * i + 1] << 16;
    }
}
__device__ __forceinline__ void load_piece(Piece<float>& p, const float* row, int at, int D) {
    if (at + 8 <= D) return load_whole(p, row + at);
#pragma unroll
    for (int i = 0; i < 8; ++i) p.v[i] = at + i < D ? row[at + i] : 0.0f;
}
__device__ __forceinline__ void no_piece(Piece<uint16_t>& p) { p.w[0] = p.w[1] = p.w[2] = p.w[3] = 0u; }
__device__ __forceinline__ void no_piece(Piece<float>& p) {
#pragma unroll
    for (int i = 0; i < 8; ++i) p.v[i] = 0.0f;
}
__device__ __forceinline__ float piece_value(const Piece<uint16_t>& p, int i) {
    return __uint_as_float(i & 1 ? p.w[i / 2] & 0xffff0000u : p.w[i / 2] << 16);
}
__device__ __forceinline__ float piece_value(const Piece<float>& p, int i) { return p.v[i]; }
template <typename TS>
struct planes_of {
    static constexpr int n = sizeof(TS) == 4 ? 3 : 1;
};
__device__ __forceinline__ void piece_planes(const Piece<uint16_t>& p, bf16x8 (&out)[1]) { __builtin_memcpy(&out[0], p.w, 16); }
__device__ __forceinline__ void piece_planes(const Piece<float>& p, bf16x8 (&out)[3]) {
    split8<3>(f32x4{p.v[0], p.v[1], p.v[2], p.v[3]}, f32x4{p.v[4], p.v[5], p.v[6], p.v[7]}, out);
}

// The 64 rows of a chunk as NT threads carry them: rows `rows` and on, and columns D
// and on, are zero.  EVEN: D is a multiple of eight, and a piece is loaded whole,
// from the last row where there is no such row and from the first columns where
// there are none, and becomes zero on its way to LDS.
template <typename TS, int W, int NT, bool EVEN>
struct Carry {
    static constexpr int CH = W / 8, N = C * CH / NT, RS = NT / CH, PL = planes_of<TS>::n;
    static_assert(N >= 1 && NT % CH == 0 && C * CH % NT == 0, "whole rounds of pieces");
    Piece<TS> p[N];
    __device__ __forceinline__ void load(int x, const TS* base, int64_t row_stride, int rows, int D) {
        const int i = (int)threadIdx.x / CH + RS * x, at = 8 * ((int)threadIdx.x % CH);
        if constexpr (EVEN) {
            load_whole(p[x], base + (at < D ? at : 0) + (uint32_t)(i < rows ? i : rows - 1) * (uint32_t)row_stride);
        } else {
            if (i < rows && at < D) load_piece(p[x], base + i * row_stride, at, D);
            else no_piece(p[x]);
        }
    }
    __device__ __forceinline__ void load(const TS* base, int64_t row_stride, int rows, int D) {
#pragma unroll
        for (int x = 0; x < N; ++x) load(x, base, row_stride, rows, D);
    }
    __device__ __forceinline__ void put(uint16_t* lds, int x) const {
        const int e = threadIdx.x + NT * x;
        bf16x8 v[PL];
        piece_planes(p[x], v);
#pragma unroll
        for (int n = 0; n < PL; ++n) *reinterpret_cast<bf16x8*>(lds + n * C * W + piece_at<W>(e / CH, e % CH)) = v[n];
    }
    __device__ __forceinline__ void store(uint16_t* lds, int rows, int D) const {
        if (!EVEN || (rows >= C && D >= W)) {          // uniform
#pragma unroll
            for (int x = 0; x < N; ++x) put(lds, x);
            return;
        }
        const bf16x8 zero = {};
        const int row = (int)threadIdx.x / CH, c = (int)threadIdx.x % CH;
#pragma unroll
        for (int x = 0; x < N; ++x) {
            if (row + RS * x < rows && 8 * c < D) {
                put(lds, x);
            } else {
#pragma unroll
                for (int n = 0; n < PL; ++n) *reinterpret_cast<bf16x8*>(lds + n * C * W + piece_at<W>(row + RS * x, c)) = zero;
            }
        }
    }
};
// BYTES that follow each other, the same way.
template <int BYTES, int NT>
struct CarryBytes {
    static constexpr int N = (BYTES / 16 + NT - 1) / NT;
    u32x4v v[N];
    __device__ __forceinline__ void load(int x, const void* from) {
        const int e = threadIdx.x + NT * x;
        if (BYTES / 16 % NT == 0 || e < BYTES / 16) v[x] = static_cast<const u32x4v*>(from)[e];
    }
    __device__ __forceinline__ void load(const void* from) {
#pragma unroll
        for (int x = 0; x < N; ++x) load(x, from);
    }
    __device__ __forceinline__ void store(void* to) const {
#pragma unroll
        for (int x = 0; x < N; ++x) {
            const int e = threadIdx.x + NT * x;
            if (e < BYTES / 16) static_cast<u32x4v*>(to)[e] = v[x];
        }
    }
};

// 64 rows, or BYTES that follow each other, from HBM to LDS without a register in
// between (16 bytes a lane, a wave's lanes one after the other).  A lane asks for
// the piece that belongs in its place; rows `rows` and on, and columns D and on, become
// zero.  What is under way has arrived after `arrived` and a barrier.
typedef __attribute__((address_space(3))) void lds_void;
typedef const __attribute__((address_space(1))) void hbm_void;
__device__ __forceinline__ void to_lds(const void* from, char* to) {
    __builtin_amdgcn_global_load_lds((hbm_void*)from, (lds_void*)to, 16, 0, 0);
}
__device__ __forceinline__ void arrived() { __builtin_amdgcn_s_waitcnt(0x0f70); }      // vmcnt(0)
__device__ const uint4 kZeros = {0u, 0u, 0u, 0u};
template <int W, int NT>
struct Direct {
    static constexpr int CH = W / 8, N = C * CH / NT;
    static_assert(N >= 1, "a piece for every thread");
    uint32_t off[N];                                   // this thread's pieces of a chunk, in bytes
    int row[N];                                        // and their rows; past the last one where there is no such column
    __device__ __forceinline__ void plan(int64_t row_stride, int D) {
#pragma unroll
        for (int x = 0; x < N; ++x) {
            const int e = threadIdx.x + NT * x, i = e / CH, c = piece_at<W>(i, e % CH) / 8 % CH;
            off[x] = 2 * ((uint32_t)i * (uint32_t)row_stride + 8 * (uint32_t)c);
            row[x] = 8 * c < D ? i : INT32_MAX;
        }
    }
    __device__ __forceinline__ void load(int x, const uint16_t* base, int rows, char* lds) const {
        const char* from = reinterpret_cast<const char*>(base) + off[x];
        if (row[x] >= rows) from = reinterpret_cast<const char*>(&kZeros);
        to_lds(from, lds + 16 * ((int)(threadIdx.x & ~63) + NT * x));
    }
};
template <int BYTES, int NT>
struct DirectBytes {
    static constexpr int N = (BYTES / 16 + NT - 1) / NT;
    static_assert(BYTES % 1024 == 0, "whole waves");
    static __device__ __forceinline__ void load(int x, const void* from, char* lds) {
        const int first = __builtin_amdgcn_readfirstlane((int)threadIdx.x & ~63) + NT * x;
        if (BYTES / 16 % NT != 0 && first >= BYTES / 16) return;       // uniform
        to_lds(static_cast<const char*>(from) + 16 * (first + ((int)threadIdx.x & 63)), lds + 16 * first);
    }
};

// A triangular matrix of 64 x 64 as left operand: six pieces [tile][32 columns] of 64
// lanes by eight values are not zero, a plane after the other.
constexpr int kTri = 6 * 64 * 8;
__device__ __forceinline__ int lower_piece(int tile, int s) { return tile < 2 ? tile : 2 * tile - 2 + s; }    // s <= tile / 2
__device__ __forceinline__ int upper_piece(int tile, int s) { return tile < 2 ? 2 * tile + s : tile + 2; }    // s >= tile / 2
template <int PL>
__device__ __forceinline__ void tri_frag(const uint16_t* lds, int piece, bf16x8 (&out)[PL]) {
#pragma unroll
    for (int n = 0; n < PL; ++n)
        out[n] = *reinterpret_cast<const bf16x8*>(lds + n * kTri + (piece * 64 + (threadIdx.x & 63)) * 8);
}

__device__ __forceinline__ int64_t at_row(const kan_heads_t& s, int64_t b, int64_t t, int64_t h) {
    return b * s.seq + t * s.row + h * s.head;
}
// Head and column tile of a scan's block: a head's blocks read the same rows, so
// they go to one XCD (blocks are dealt to the eight of them in turn) and its L2
// (the backward scan of 4 x 4096 x 16 x 128 bf16 takes 393 us without this and 369
// with it, the forward scan of 8 x 4096 338 and 336).
__device__ __forceinline__ void head_and_tile(int heads, int tiles, int& head, int& tile) {
    const int group = (int)blockIdx.x / (8 * tiles), at = (int)blockIdx.x % (8 * tiles);
    const int n = heads - 8 * group < 8 ? heads - 8 * group : 8;
    head = 8 * group + at % n;
    tile = at / n;
}
__device__ __forceinline__ int length_of(const DeltaArgs& a, int64_t b, int64_t T) {
    if (!a.lengths) return (int)T;
    const int n = a.lengths[b];
    return n < 0 ? 0 : n > T ? (int)T : n;
}
// exp(c_i - c_j) by the hardware's 2^x; below 2^-126 it is 0.
__device__ __forceinline__ float decay(const float* row, int i, int j) {
    return __builtin_amdgcn_exp2f((row[kHi * C + i] - row[kHi * C + j]) + (row[kLo * C + i] - row[kLo * C + j]));
}
// exp(c_63), what a chunk leaves of the state before it
__device__ __forceinline__ float whole_decay(const float* row) {
    return __builtin_amdgcn_exp2f(row[kHi * C + C - 1] + row[kLo * C + C - 1]);
}

// ---- a chunk's rows among themselves -------------------------------------------

// Factors that make rows unit vectors (sums over the planes' values).
template <int PL, int W, int NT>
__device__ __forceinline__ void unit_factors(const uint16_t* lds, float* factor) {
    constexpr int PER = NT / C;                        // threads of a row
    const int row = threadIdx.x / PER;
    float n = 0.0f;
#pragma unroll
    for (int c = threadIdx.x % PER; c < W / 8; c += PER) {
        float x[8];
#pragma unroll
        for (int z = 0; z < PL; ++z) {
            uint32_t w[4];
            __builtin_memcpy(w, lds + z * C * W + piece_at<W>(row, c), 16);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float v = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
                x[i] = z ? x[i] + v : v;
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) n = __builtin_fmaf(x[i], x[i], n);
    }
#pragma unroll
    for (int o = 1; o < PER; o <<= 1) n += __shfl_xor(n, o, 64);
    if (threadIdx.x % PER == 0) factor[row] = 1.0f / sqrtf(n + kUnitEps);
}

// float32 products of 16 x 16 blocks for the triangular solution: lane (gq, m) has
// four values 4 gq .. + 3 of the contracted index.
__device__ __forceinline__ void mma_f32(f32x4& acc, const f32x4& a, const f32x4& b) {
#pragma unroll
    for (int j = 0; j < 4; ++j) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], acc, 0, 0, 0);
}

// G in place of A (strictly lower, LDS pitch LC): G = A - A diag(beta) G.
__device__ __forceinline__ void solve(float* A, const float* beta) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, m = lane & 15, gq = lane >> 4;
    // the diagonal blocks of 16, a wave each, column m to a lane ...
    {
        float h[16];                                   // beta_k G[k][m]
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float* Ai = A + (16 * wave + i) * LC + 16 * wave;
            float v = Ai[m];
#pragma unroll
            for (int k = 0; k < i; ++k) v = __builtin_fmaf(-Ai[k], h[k], v);
            h[i] = v * beta[16 * wave + i];
            if (gq == 0) Ai[m] = v;
        }
    }
    __syncthreads();
    // ... and the blocks below, a row of blocks after the other: wave j has block j,
    // R = A_ij - sum over k of A_ik diag(beta) G_kj,  G_ij = R - G_ii diag(beta) R
    const int j = 16 * wave + m;
    for (int it = 1; it < 4; ++it) {
        f32x4 R = zero4();
        auto scaled = [&](int kt) {
            f32x4 v;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int k = 16 * kt + 4 * gq + x;
                v[x] = -beta[k] * A[k * LC + j];
            }
            return v;
        };
        if (wave < it) {
            for (int kt = wave; kt < it; ++kt) mma_f32(R, ld4(A + (16 * it + m) * LC + 16 * kt + 4 * gq), scaled(kt));
#pragma unroll
            for (int x = 0; x < 4; ++x) R[x] += A[(16 * it + 4 * gq + x) * LC + j];
        }
        __syncthreads();                               // A_ik has been read
        if (wave < it) {
#pragma unroll
            for (int x = 0; x < 4; ++x) A[(16 * it + 4 * gq + x) * LC + j] = R[x];
            mma_f32(R, ld4(A + (16 * it + m) * LC + 16 * it + 4 * gq), scaled(it));
#pragma unroll
            for (int x = 0; x < 4; ++x) A[(16 * it + 4 * gq + x) * LC + j] = R[x];
        }
    }
    __syncthreads();
}

// Pieces of a triangular matrix (LDS pitch LC) or of its transpose, as operands.
template <int PL, bool TRANSPOSED>
__device__ __forceinline__ void write_tri(const float* X, uint16_t* out, int nt) {
    for (int e = threadIdx.x; e < 6 * 64; e += nt) {
        const int piece = e >> 6, lane = e & 63;
        int tile, s;
        if (TRANSPOSED) tile = piece < 4 ? piece >> 1 : piece - 2, s = piece < 4 ? piece & 1 : 1;
        else tile = piece < 2 ? piece : (piece >> 1) + 1, s = piece < 2 ? 0 : piece & 1;
        const int i = row_of(tile, lane & 15), j = 32 * s + 8 * (lane >> 4);
        f32x4 v[2];
        if (TRANSPOSED) {
#pragma unroll
            for (int x = 0; x < 8; ++x) v[x >> 2][x & 3] = X[(j + x) * LC + i];
        } else {
            v[0] = ld4(X + i * LC + j), v[1] = ld4(X + i * LC + j + 4);
        }
        bf16x8 p[PL];
        split8<PL>(v[0], v[1], p);
#pragma unroll
        for (int n = 0; n < PL; ++n) *reinterpret_cast<bf16x8*>(out + n * kTri + e * 8) = p[n];
    }
}

constexpr int PREP_NT = 256;
template <typename TS, int DKP>
constexpr int prep_bytes() {                           // of K, then of A and P in its place
    constexpr int rows = 2 * planes_of<TS>::n * C * DKP, pairs = 8 * C * LC;
    return rows > pairs ? rows : pairs;
}
// Chunk n of sequence b for the heads that share a key: row fields, G and P (BWD: G
// and the transposes).  The products K K^T and Q K^T are the heads' own; rows of Q
// are left operands straight from HBM.  SHARED: a key has several heads; the loop over
// them keeps the products in registers, which one head need not pay for (8 x 4096 x
// 16 x 128 bf16 forward: 139 us with it, 118 without).
template <typename TS, int DKP, bool BWD, bool SHARED>
__global__ void __launch_bounds__(PREP_NT) delta_prep_kernel(kan_delta_desc_t d, DeltaPlan p, DeltaArgs a, char* ws) {
    extern __shared__ __align__(16) char lds[];
    constexpr int PL = planes_of<TS>::n, STEPS = DKP / 32;
    uint16_t* const K = reinterpret_cast<uint16_t*>(lds);          // [PL][64][DKP]
    float* const A = reinterpret_cast<float*>(lds);                // [64][LC], G in the end
    float* const P = A + C * LC;
    float* const row = reinterpret_cast<float*>(lds + prep_bytes<TS, DKP>());      // [8][64]
    const int64_t n = blockIdx.x % (unsigned)p.chunks, bk = blockIdx.x / (unsigned)p.chunks;
    const int64_t b = bk / d.Hk, hk = bk % d.Hk;
    const int rows = length_of(a, b, d.T) - (int)n * C, share = SHARED ? (int)(d.Hv / d.Hk) : 1;
    if (rows <= 0) return;                             // uniform
    const int64_t t0 = n * C;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, m = lane & 15, gq = lane >> 4;
    const int im = 16 * wave + m, i0 = 16 * wave + 4 * gq;
    const TS* const q = static_cast<const TS*>(a.q) + at_row(d.q, b, t0 + (im < rows ? im : 0), hk);
    Piece<TS> qp[STEPS];
    {
        Carry<TS, DKP, PREP_NT, false> k;
        k.load(static_cast<const TS*>(a.k) + at_row(d.k, b, t0, hk), d.k.row, rows, (int)d.Dk);
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int at = 32 * s + 8 * gq;
            if (im < rows && at < d.Dk) load_piece(qp[s], q, at, (int)d.Dk);
            else no_piece(qp[s]);
        }
        k.store(K, rows, (int)d.Dk);
    }
    if (tid < C) row[kNk * C + tid] = row[kNq * C + tid] = 1.0f;
    __syncthreads();
    if (d.flags & KAN_DELTA_UNIT) {
        unit_factors<PL, DKP, PREP_NT>(K, row + kNk * C);
        float sq = 0.0f;
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
#pragma unroll
            for (int j = 0; j < 8; ++j) sq = __builtin_fmaf(piece_value(qp[s], j), piece_value(qp[s], j), sq);
        sq += __shfl_xor(sq, 16, 64);
        sq += __shfl_xor(sq, 32, 64);
        if (gq == 0) row[kNq * C + im] = 1.0f / sqrtf(sq + kUnitEps);
    }
    // this wave's 16 rows of K K^T and Q K^T
    f32x4 kk[4], qk[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) kk[x] = qk[x] = zero4();
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        bf16x8 ka[PL], qa[PL];
        row_frag<PL, DKP>(K, im, 4 * s + gq, ka);
        piece_planes(qp[s], qa);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            if (x > wave) break;
            bf16x8 kb[PL];
            row_frag<PL, DKP>(K, 16 * x + m, 4 * s + gq, kb);
            mma<PL, PL>(kk[x], ka, kb);
            mma<PL, PL>(qk[x], qa, kb);
        }
    }
    __syncthreads();                                   // the unit factors are there
#pragma unroll 1
    for (int z = 0; z < share; ++z) {
        const int64_t h = hk * share + z, bh = b * d.Hv + h, ch = bh * p.chunks + n;
        if (wave == 0) {
            float g = 0.0f, beta = 0.0f;
            if (lane < rows) {
                g = a.g[(b * d.T + t0 + lane) * d.Hv + h];
                beta = a.beta[(b * d.T + t0 + lane) * d.Hv + h];
                // finite, for differences of sums; 0 also after what growth a float holds; a NaN stays
                g = g < -1024.0f ? -1024.0f : g;
            }
            double c = (double)g * 1.4426950408889634;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const double before = __shfl_up(c, o, 64);
                if (lane >= o) c += before;
            }
            const float hi = (float)c, lo = hi - hi == 0.0f ? (float)(c - (double)hi) : 0.0f;
            const float from = __builtin_amdgcn_exp2f(hi + lo), nk = row[kNk * C + lane];
            row[kHi * C + lane] = hi;
            row[kLo * C + lane] = lo;
            row[kBeta * C + lane] = beta;
            row[kFk * C + lane] = from * nk;
            row[kTk * C + lane] = __builtin_amdgcn_exp2f((float)(__shfl(c, 63, 64) - c)) * nk;
            row[kFq * C + lane] = from;
        }
        __syncthreads();                               // and K, or the matrices of the head before, are done with
        {
            const f32x4 hi = ld4(row + kHi * C + i0), lo = ld4(row + kLo * C + i0);
            const f32x4 ni = ld4(row + kNk * C + i0), nq = d.scale * ld4(row + kNq * C + i0);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                if (x > (wave | 1)) break;             // blocks that no piece reaches
                const int j = 16 * x + m;
                const float nj = row[kNk * C + j], hj = row[kHi * C + j], lj = row[kLo * C + j];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const int i = i0 + y;
                    const float D = nj * __builtin_amdgcn_exp2f((hi[y] - hj) + (lo[y] - lj));
                    A[i * LC + j] = j < i ? kk[x][y] * (D * ni[y]) : 0.0f;
                    P[i * LC + j] = j <= i ? qk[x][y] * (D * nq[y]) : 0.0f;
                }
            }
            if (m == 0) st4(row + kFq * C + i0, ld4(row + kFq * C + i0) * nq);
        }
        __syncthreads();
        float* const out_row = reinterpret_cast<float*>(ws + p.off_rows) + ch * kFields * C;
        for (int i = tid; i < kFields * C; i += PREP_NT) out_row[i] = row[i];
        uint16_t* const mats = reinterpret_cast<uint16_t*>(ws + p.off_mats + ch * p.mats);
        if (BWD) write_tri<3, true>(P, mats + 6 * kTri, PREP_NT);
        else write_tri<3, false>(P, mats + 3 * kTri, PREP_NT);
        solve(A, row + kBeta * C);
        write_tri<3, false>(A, mats, PREP_NT);
        if (BWD) write_tri<3, true>(A, mats + 3 * kTri, PREP_NT);
        if (z + 1 < share) __syncthreads();            // the rows' fields are done with
    }
}

// ---- along a sequence -------------------------------------------------------------

enum Pass { kForward, kStates, kRuns, kBack };

constexpr int kan_delta_halves(int dkp, int groups) { return dkp >= 64 && groups == 2 ? 2 : 1; }

// How a scan's block is laid out.  A wave has 16 columns of the state.  In blocks
// of two groups with room for it in Dk it has half of the state's rows, and a pair
// of waves shares the columns: what each contracts over its rows of the state is
// added to the other's through LDS, and all four SIMDs have a wave.  LDS and
// registers leave most scans one block a compute unit.
template <typename TS, int DKP, int GROUPS, int PASS, bool EVEN>
struct Scan {
    static constexpr int PL = planes_of<TS>::n, NP = 3;          // planes of rows, and of the floats behind y
    static constexpr bool FWD = PASS == kForward, BACK = PASS == kBack;
    static constexpr int HALVES = kan_delta_halves(DKP, GROUPS), NT = 64 * GROUPS * HALVES, W = 16 * GROUPS;
    static constexpr int DT = DKP / 16 / HALVES, STEPS = DKP / 32 / HALVES;     // tiles and operands of a wave's state
    // bfloat16 rows are operands as they stand: they go to LDS by themselves, into
    // a second buffer.  Others pass through registers into one buffer.
    static constexpr bool DIRECT = PL == 1 && EVEN;
    // float32 has no room for P, which the waves then read from the workspace
    static constexpr bool P_LDS = (FWD || BACK) && PL == 1;
    static constexpr int MATS = (P_LDS ? 6 : 3) * kTri;   // G, P (or transposed)
    static constexpr int ROWS = PL * C * DKP;
    static constexpr int K = 0, Q = K + ROWS * 2, V = Q + (FWD || BACK ? ROWS * 2 : 0);        // offsets in bytes
    static constexpr int FIELDS = V + (BACK ? PL * C * W * 2 : DIRECT ? C * W * 2 : 0);
    static constexpr int BUF = FIELDS + kFields * C * 4;
    static constexpr int SLOT = 4 * 64 * 16, SLOTS = HALVES == 2 ? 2 * GROUPS * SLOT : 0;      // a slot: four tiles of a wave
    // the matrices too have a second buffer where there is room, and go there directly
    static constexpr bool MATS_DIRECT = DIRECT && 2 * (BUF + MATS * 2) + SLOTS <= 160 * 1024;
    static constexpr int G = (DIRECT ? 2 : 1) * BUF, G_BUF = MATS_DIRECT ? MATS * 2 : 0, P = 3 * kTri * 2;
    static constexpr int SLOT0 = G + MATS * 2 + G_BUF, LDS = SLOT0 + SLOTS;
};

// The products of a scan.  Operands are loaded a group ahead of the instructions
// that use them, and a group goes plane by plane over its tiles, so that an
// instruction never waits for the one before it.  The fences hold the compiler to
// that order.  They are worth 3 to 7 hundredths of a float32 backward pass with keys
// of 128 (8 x 4096 x 16 heads: 2897 us with them, 3089 without) and cost a few
// hundredths in most others (bf16: forward 497 and 489, backward 1582 and 1541).
#define KAN_FENCE() __builtin_amdgcn_sched_barrier(0)

// acc[t] += a[t] b for T tiles
template <int T, int NA, int NB>
__device__ __forceinline__ void mma_tiles(f32x4* acc, const bf16x8 (*a)[NA], const bf16x8 (&b)[NB]) {
    constexpr int N = NA > NB ? NA : NB;
#pragma unroll
    for (int place = N - 1; place >= 0; --place)
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (place - i >= 0 && place - i < NB)
#pragma unroll
                for (int t = 0; t < T; ++t)
                    acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[t][i], b[place - i], acc[t], 0, 0, 0);
}
// acc[t] += b a[t]: the result transposed
template <int T, int NA, int NB>
__device__ __forceinline__ void mma_tiles_t(f32x4* acc, const bf16x8 (*a)[NA], const bf16x8 (&b)[NB]) {
    constexpr int N = NA > NB ? NA : NB;
#pragma unroll
    for (int place = N - 1; place >= 0; --place)
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (place - i >= 0 && place - i < NB)
#pragma unroll
                for (int t = 0; t < T; ++t)
                    acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[place - i], a[t][i], acc[t], 0, 0, 0);
}

// T tiles of rows from `first` on, in pieces 4 s .. of K or Q.
template <int T, int PL, int DKP>
__device__ __forceinline__ void load_rows(const uint16_t* lds, int s, int first, bf16x8 (*f)[PL]) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int t = 0; t < T; ++t) row_frag<PL, DKP>(lds, row_of((first + t) & 3, lane & 15), 4 * s + (lane >> 4), f[t]);
}
// The tiles of rows that have 32 columns s of a triangular matrix: lower, all four
// for s = 0 and the last two for s = 1; upper, the first two for s = 0, all for s = 1.
template <int PL, bool UPPER, bool ALL>
__device__ __forceinline__ void load_tri(const uint16_t* lds, bf16x8 (*f)[PL]) {
#pragma unroll
    for (int t = 0; t < (ALL ? 4 : 2); ++t)
        tri_frag<PL>(lds, UPPER ? upper_piece(t, ALL ? 1 : 0) : lower_piece(ALL ? t : t + 2, ALL ? 0 : 1), f[t]);
}
// Columns of K or Q for the tiles 2 g, 2 g + 1 of the state, rows 32 s and on.
template <int PL, int DKP>
__device__ __forceinline__ void load_cols(const uint16_t* lds, int g, int s, bf16x8 (*f)[PL]) {
    const int m = threadIdx.x & 15;
#pragma unroll
    for (int x = 0; x < 2; ++x) col_frag<PL, DKP>(lds, s, 4 * g + (m & 3), x, f[x]);
}
__device__ __forceinline__ f32x4 at_rows(const float* row, int field, int t) {
    return ld4(row + field * C + row_of(t, 4 * ((threadIdx.x & 63) >> 4)));
}

// So many vector instructions beside every matrix instruction of a region.
template <int N, int VALU>
__device__ __forceinline__ void beside() {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, VALU, 0);
    }
}

// ks[t] += rows of K times a wave's part of the state, of which NS planes are kept
// in `sp`.  `last` loads what comes next, `ahead` parts of the next chunk.
template <typename L, int DKP, int NS, typename Ahead, typename Last>
__device__ __forceinline__ void rows_by_state(const uint16_t* K, int step0, const f32x4* S, f32x4 (&ks)[4],
                                              bf16x8 (*sp)[NS], Ahead ahead, Last last) {
    constexpr int PL = L::PL, TG = PL == 1 ? 4 : 2, PARTS = 4 / TG;
    bf16x8 f[2][TG][PL], sb[2][3];
    load_rows<TG, PL, DKP>(K, step0, 0, f[0]);
    split8<3>(S[0], S[1], sb[0]);
#pragma unroll
    for (int g = 0; g < L::STEPS * PARTS; ++g) {
        const int s = g / PARTS, at = g % PARTS * TG;
        if (g + 1 < L::STEPS * PARTS)
            load_rows<TG, PL, DKP>(K, step0 + (g + 1) / PARTS, (g + 1) % PARTS * TG, f[(g + 1) & 1]);
        else
            last();
        KAN_FENCE();
        mma_tiles<TG, PL, 3>(ks + at, f[g & 1], sb[s & 1]);
        if (g % PARTS == 0) {
#pragma unroll
            for (int z = 0; z < NS; ++z) sp[s][z] = sb[s & 1][z];
            if (s + 1 < L::STEPS) {
                split8<3>(S[2 * s + 2], S[2 * s + 3], sb[(s + 1) & 1]);
                beside<12, 4>();
            }
        }
        KAN_FENCE();
        if (g == 0) ahead(1);                          // parts 1 and 2 of what comes
        if (g == L::STEPS * PARTS / 2) ahead(2);
    }
}
// o[t] += the transposed product of rows of Q, tiles from `first` on, with the
// state's planes; beside it goes the work of `more`, in four parts.
template <typename L, int DKP, typename More, typename Last>
__device__ __forceinline__ void state_by_rows(const uint16_t* Q, int step0, int first, const bf16x8 (*sp)[L::NP],
                                              f32x4 (&o)[4], bf16x8 (*f)[L::PL == 1 ? 4 : 2][L::PL], More more, Last last) {
    constexpr int PL = L::PL, NP = L::NP, TG = PL == 1 ? 4 : 2, PARTS = 4 / TG, N = L::STEPS * PARTS;
#pragma unroll
    for (int g = 0; g < N; ++g) {
        if (g + 1 < N) load_rows<TG, PL, DKP>(Q, step0 + (g + 1) / PARTS, first + (g + 1) % PARTS * TG, f[(g + 1) & 1]);
        else last();
        KAN_FENCE();
        mma_tiles_t<TG, PL, NP>(o + g % PARTS * TG, f[g & 1], sp[g / PARTS]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i * N / 4 == g) more(i);
        beside<8, 4>();
        KAN_FENCE();
    }
}
// A wave's tiles to its slot, and the partner's added.
__device__ __forceinline__ void give_tiles(char* slot, const f32x4* v, int n) {
#pragma unroll
    for (int t = 0; t < n; ++t) st4(reinterpret_cast<float*>(slot) + (t * 64 + (threadIdx.x & 63)) * 4, v[t]);
}
__device__ __forceinline__ void add_tiles(const char* slot, f32x4* v, int n) {
#pragma unroll
    for (int t = 0; t < n; ++t) v[t] = v[t] + ld4(reinterpret_cast<const float*>(slot) + (t * 64 + (threadIdx.x & 63)) * 4);
}

// Along the sequences of a head: the state stays in registers from the start to
// the end, and what a wave computes of a chunk's rows in its columns is an
// operand of its next product as it stands.  The left operands (K, Q, G, P) are
// the same for the block's waves and come through LDS; the next chunk's are on
// their way from HBM meanwhile.  PASS kStates: keeps the chunks' first states and w
// for the backward pass and writes no rows.
//
// Where heads are too few to fill the GPU their chunks are cut into segments.  A
// segment takes the state before it to M S + B; PASS kRuns finds M, which is what
// becomes of the columns of the identity without values, and B, which is what
// becomes of no state; the starts of the segments follow from these one after the
// other (delta_link_kernel), and the pass itself runs all segments at once.
template <typename TS, int DKP, int GROUPS, int PASS, bool EVEN>
__global__ void __launch_bounds__((Scan<TS, DKP, GROUPS, PASS, EVEN>::NT))
    delta_scan_kernel(kan_delta_desc_t d, DeltaPlan p, DeltaArgs a, char* ws) {
    typedef Scan<TS, DKP, GROUPS, PASS, EVEN> L;
    extern __shared__ __align__(16) char lds[];
    constexpr bool FWD = L::FWD, DIRECT = L::DIRECT;
    constexpr int PL = L::PL, NP = L::NP, NT = L::NT, W = L::W, DT = L::DT, HALVES = L::HALVES, OWN = 4 / HALVES;
    constexpr bool RUNS = PASS == kRuns;
    const int vtiles = (int)((d.Dv + W - 1) / W), mtiles = RUNS ? (DKP + W - 1) / W : 0;
    int head, tile;
    head_and_tile((int)p.heads * (RUNS ? p.runs : p.segs), vtiles + mtiles, head, tile);
    const int seg = head / (int)p.heads;
    const int64_t bh = head % (int)p.heads, b = bh / d.Hv, h = bh % d.Hv, hk = h / (d.Hv / d.Hk);
    const int tid = threadIdx.x, lane = tid & 63, m = lane & 15, gq = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), half = wave % HALVES;
    const bool of_m = RUNS && tile >= vtiles;                      // columns of the identity
    if (of_m && seg == 0) return;                                  // the first segment starts from h0
    const int nb = (of_m ? tile - vtiles : tile) * W, n0 = nb + 16 * (wave / HALVES);   // the block's and this wave's first column
    const int Dk = (int)d.Dk, Dv = (int)d.Dv, len = length_of(a, b, d.T), all = (len + C - 1) / C;
    // this segment's chunks
    const int first = seg * p.seg_chunks, chunks = all < first + p.seg_chunks ? all : first + p.seg_chunks;
    const bool mine = n0 + m < (of_m ? Dk : Dv);
    const int x0 = half * DT;                                      // this wave's first tile of the state
    const float* start = a.h0 ? a.h0 + bh * Dk * Dv : nullptr;     // [Dk][Dv], or of the workspace [dkp][dvp]
    int start_row = Dv;
    if (seg > 0) {
        start = RUNS ? nullptr : reinterpret_cast<const float*>(ws + p.off_starts) + (seg * p.heads + bh) * DKP * p.dvp;
        start_row = p.dvp;
    }
    f32x4 S[DT];
#pragma unroll
    for (int x = 0; x < DT; ++x)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int dd = row_of(x0 + x, 4 * gq) + j;
            S[x][j] = of_m ? (dd == n0 + m && mine ? 1.0f : 0.0f)
                           : start && dd < Dk && mine ? start[(int64_t)dd * start_row + n0 + m] : 0.0f;
        }
    const TS* const k_base = static_cast<const TS*>(a.k) + at_row(d.k, b, 0, hk);
    const TS* const q_base = static_cast<const TS*>(a.q) + at_row(d.q, b, 0, hk);
    const TS* const v_base = static_cast<const TS*>(a.v) + at_row(d.v, b, 0, h);      // not used where of_m
    TS* const y_base = static_cast<TS*>(a.y) + (b * d.T * d.Hv + h) * Dv;
    const float* const rows_base = reinterpret_cast<const float*>(ws + p.off_rows) + bh * p.chunks * kFields * C;
    const char* const mats_base = ws + p.off_mats + bh * p.chunks * p.mats;
    Carry<TS, DKP, NT, EVEN> ck, cq;
    CarryBytes<L::MATS * 2, NT> cm;
    CarryBytes<kFields * C * 4, NT> cr;
    Direct<DKP, NT> xk, xq;
    Direct<W, NT> xv;
    if (DIRECT) {
        xk.plan(d.k.row, Dk);
        if (FWD) xq.plan(d.q.row, Dk);
        xv.plan(d.v.row, of_m ? 0 : Dv - nb);          // no values: zeros
    }
    // rows of a chunk lie at most 2^32 bytes apart: a lane's part of an address
    const uint32_t v_row = (uint32_t)d.v.row, y_row = (uint32_t)(d.Hv * Dv), column = mine && !of_m ? n0 + m : 0;
    const uint32_t y_off = (uint32_t)row_of(0, m) * y_row + n0 + 4 * gq;
    const uint32_t s_off = 8 * gq * (uint32_t)p.dvp + n0 + m;
    TS vn[4][4];
    // Chunk n on its way to LDS, or to registers.  Through registers it goes a few
    // loads at a time between the products (1 x 32768 x 8 x 128 float32: scan 428 us
    // at once, 386 in eight parts); directly to LDS all of it at once, since loads
    // between the products hold those up as well (8 x 4096 x 16 x 128 bf16: 336 us at
    // once, 345 in parts; the states of 4 x 4096 257 and 323).
    constexpr int PARTS = DIRECT ? 1 : 8;
    auto fetch = [&](int part, int n) {
        const int64_t t0 = (int64_t)n * C;
        const int rows = len - n * C;
        char* const to = lds + (DIRECT ? (n & 1) * L::BUF : 0);
        const char* const mats = mats_base + n * p.mats;
        const float* const fields = rows_base + (int64_t)n * kFields * C;
        constexpr int NK = ck.N, NQ = FWD ? NK : 0, NV = DIRECT ? xv.N : 16, NM = cm.N, NF = cr.N;
        constexpr int ALL = NK + NQ + NV + NM + NF;
#pragma unroll
        for (int j = 0; j < ALL; ++j) {
            if (j * PARTS / ALL != part) continue;
            const int q = j - NK, v = q - NQ, x = v - NV, f = x - NM;
            if (j < NK) {
                if constexpr (DIRECT) xk.load(j, k_base + t0 * d.k.row, rows, to + L::K);
                else ck.load(j, k_base + t0 * d.k.row, d.k.row, rows, Dk);
            } else if (q < NQ) {
                if constexpr (DIRECT) xq.load(q, q_base + t0 * d.q.row, rows, to + L::Q);
                else cq.load(q, q_base + t0 * d.q.row, d.q.row, rows, Dk);
            } else if (v < NV) {
                if constexpr (DIRECT) {
                    xv.load(v, v_base + t0 * d.v.row + nb, rows, to + L::V);
                } else {
                    const int i = row_of(v / 4, v % 4) + 8 * gq;
                    vn[v / 4][v % 4] = (v_base + t0 * d.v.row)[(uint32_t)(i < rows ? i : rows - 1) * v_row + column];
                }
            } else if (x < NM) {
                if constexpr (L::MATS_DIRECT)
                    DirectBytes<L::MATS * 2, NT>::load(x, mats, lds + L::G + (n & 1) * L::G_BUF);
                else cm.load(x, mats);
            } else {
                if constexpr (DIRECT) DirectBytes<kFields * C * 4, NT>::load(f, fields, to + L::FIELDS);
                else cr.load(f, fields);
            }
        }
    };
    char* const my_slot = lds + L::SLOT0 + wave * L::SLOT;
    char* const other_slot = lds + L::SLOT0 + (wave ^ 1) * L::SLOT;
    // The rows of a chunk are stored in the next one's time: what waits for the
    // chunk's arrival waits for stores under way as well.  A pair of waves has two
    // tiles of rows each, o[0] and o[1] of tiles 2 half, 2 half + 1.
    f32x4 o[4], w[4];
    auto put_rows = [&](int n) {
        TS* const out = y_base + (int64_t)n * C * y_row;
        const int rows = len - n * C;
        if (HALVES == 2) add_tiles(my_slot, o, OWN);
#pragma unroll
        for (int l = 0; l < OWN; ++l) {
            const int t = HALVES == 2 ? 2 * half + l : l;
            if (row_of(t, m) >= rows) continue;
            TS* y = out + (uint32_t)row_of(t, 0) * y_row + y_off;
            if (n0 + 16 <= Dv) {                       // uniform
                const float v[4] = {o[l][0], o[l][1], o[l][2], o[l][3]};
                store_vec<4>(y, v);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (n0 + 4 * gq + j < Dv) put(y + j, o[l][j]);
            }
        }
    };
    if (first < chunks) {
#pragma unroll
        for (int part = 0; part < PARTS; ++part) fetch(part, first);
    }
    for (int n = first; n < chunks; ++n) {
        const int64_t ch = bh * p.chunks + n;
        const int rows = len - n * C;
        char* const buf = lds + (DIRECT ? (n & 1) * L::BUF : 0);
        if (DIRECT) arrived();
        __syncthreads();                               // direct: the chunk is there; else: LDS is free
        if (!DIRECT) {
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) w[t][j] = !of_m && row_of(t, j) + 8 * gq < rows ? load_f(&vn[t][j], 0) : 0.0f;
            ck.store(reinterpret_cast<uint16_t*>(lds + L::K), rows, Dk);
            if (FWD) cq.store(reinterpret_cast<uint16_t*>(lds + L::Q), rows, Dk);
            cr.store(lds + L::FIELDS);
        }
        if constexpr (!L::MATS_DIRECT) cm.store(lds + L::G);
        if (!DIRECT) __syncthreads();
        // nothing may be on its way to LDS when the block ends
        auto ahead = [&](int part) {
            if (part < PARTS && (!DIRECT || n + 1 < chunks)) fetch(part, n + 1 < chunks ? n + 1 : n);
        };
        ahead(0);
        if (FWD && n > first) put_rows(n - 1);
        const uint16_t* const K = reinterpret_cast<const uint16_t*>(buf + L::K);       // [PL][64][DKP]
        const uint16_t* const Q = reinterpret_cast<const uint16_t*>(buf + L::Q);       // forward alone
        const uint16_t* const V = reinterpret_cast<const uint16_t*>(buf + L::V);       // [64][W], direct alone
        const float* const row = reinterpret_cast<const float*>(buf + L::FIELDS);      // [8][64]
        const uint16_t* const G = reinterpret_cast<const uint16_t*>(lds + L::G + (n & 1) * L::G_BUF);  // [3][kTri]
        const uint16_t* const P = G + 3 * kTri;                                        // [NP][kTri], forward alone
        if (PASS == kStates) {
            float* out = reinterpret_cast<float*>(ws + p.off_S) + ch * DKP * p.dvp;
#pragma unroll
            for (int x = 0; x < DT; ++x)
#pragma unroll
                for (int j = 0; j < 4; ++j) (out + row_of(x0 + x, j) * p.dvp)[s_off] = S[x][j];
        }
        f32x4 fk[4], beta[4], tk[4];                   // the rows' factors, on their way meanwhile
        float fq[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            fk[t] = at_rows(row, kFk, t);
            beta[t] = at_rows(row, kBeta, t);
            tk[t] = at_rows(row, kTk, t);
            fq[t] = FWD ? row[kFq * C + row_of((t + 2 * half) & 3, m)] : 0.0f;
        }
        const float whole = whole_decay(row);
        // K S
        constexpr int TG = PL == 1 ? 4 : 2, NS = FWD ? NP : 1;
        f32x4 ks[4];
        bf16x8 sp[L::STEPS][NS], f[2][TG][PL], ga[4][3], gb[2][3];
#pragma unroll
        for (int t = 0; t < 4; ++t) ks[t] = o[t] = zero4();
        rows_by_state<L, DKP, NS>(K, half * L::STEPS, S, ks, sp, ahead, [&] {
            if constexpr (DIRECT) {
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                        (lds_s16x4*)(V + piece_at<W>(row_of(t, 4 * gq) + (m >> 2), 2 * (wave / HALVES) + ((m & 3) >> 1)) +
                                     4 * (m & 1)));
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[t][j] = __uint_as_float((uint32_t)(uint16_t)v[j] << 16);
                }
            }
            if (FWD) load_rows<TG, PL, DKP>(Q, half * L::STEPS, 2 * half, f[0]);
            if (L::MATS_DIRECT) load_tri<3, false, true>(G, ga);
        });
        ahead(3);
        if (HALVES == 2) give_tiles(my_slot, ks, 4);
        if (HALVES == 2 || !L::MATS_DIRECT) __syncthreads();           // G and P are there, and the partner's part
        if (HALVES == 2) add_tiles(other_slot, ks, 4);
        // Q S (transposed: lanes have columns of one row), and e, an operand by planes
        f32x4 be[4];
        bf16x8 eb[2][3];
        auto errors = [&](int part) {
            if (part < 2) {
#pragma unroll
                for (int t = 2 * part; t < 2 * part + 2; ++t) {
                    w[t] = w[t] - fk[t] * ks[t];       // e
                    be[t] = beta[t] * w[t];
                }
            } else {
                split8<3>(be[2 * part - 4], be[2 * part - 3], eb[part - 2]);
            }
        };
        if (!L::MATS_DIRECT) load_tri<3, false, true>(G, ga);
        if constexpr (FWD) {
            state_by_rows<L, DKP>(Q, half * L::STEPS, 2 * half, sp, o, f, errors, [&] { load_tri<3, false, false>(G, gb); });
        } else {
            load_tri<3, false, false>(G, gb);
#pragma unroll
            for (int i = 0; i < 4; ++i) errors(i);
        }
        ahead(4);
        // P for this wave's tiles: all of them, or the first two or the last two
        bf16x8 pa[4][NP], pb[2][NP];
        const uint16_t* const p_at = L::P_LDS ? P : reinterpret_cast<const uint16_t*>(mats_base + n * p.mats) + 3 * kTri;
        if (FWD && HALVES == 1) {
            load_tri<NP, false, true>(p_at, pa);
            load_tri<NP, false, false>(p_at, pb);
        } else if (FWD) {
#pragma unroll
            for (int l = 0; l < 2; ++l) {
                tri_frag<NP>(p_at, half ? lower_piece(2 + l, 0) : l, pa[l]);
                if (half) tri_frag<NP>(p_at, lower_piece(2 + l, 1), pb[l]);
            }
        }
        KAN_FENCE();
        f32x4 ge[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) ge[t] = zero4();
        mma_tiles<4, 3, 3>(ge, ga, eb[0]);
        mma_tiles<2, 3, 3>(ge + 2, gb, eb[1]);
#pragma unroll
        for (int x = 0; x < DT; ++x) S[x] = whole * S[x];
        if (FWD) {
#pragma unroll
            for (int l = 0; l < 4; ++l) o[l] = o[l] * fq[l];
        }
        // columns of K: all of them at once, or two groups ahead
        constexpr int GROUP_N = 2 * L::STEPS, AHEAD = PL == 1 ? GROUP_N : 2;
        bf16x8 kc[AHEAD][2][PL];
#pragma unroll
        for (int g = 0; g < AHEAD; ++g) load_cols<PL, DKP>(K, half * L::STEPS + g / 2, g & 1, kc[g]);
        KAN_FENCE();
        ahead(5);
        if (FWD && HALVES == 2) give_tiles(other_slot, o + 2, 2);      // read before; the partner adds it after the next barrier
        f32x4 u[4];
        bf16x8 ub[2][3], uo[2][NP];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            w[t] = w[t] - ge[t];
            u[t] = beta[t] * w[t];
        }
        if (FWD) {
            split8<NP>(u[0], u[1], uo[0]);
            split8<NP>(u[2], u[3], uo[1]);
            KAN_FENCE();
            if (HALVES == 2) {
                mma_tiles_t<2, NP, NP>(o, pa, uo[0]);
                if (half) mma_tiles_t<2, NP, NP>(o, pb, uo[1]);
            } else {
                mma_tiles_t<4, NP, NP>(o, pa, uo[0]);
                mma_tiles_t<2, NP, NP>(o + 2, pb, uo[1]);
            }
        } else if (PASS == kStates) {
            float* out = reinterpret_cast<float*>(ws + p.off_w) + ch * C * p.dvp;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                if (HALVES == 2 && t / 2 != half) continue;            // uniform
#pragma unroll
                for (int j = 0; j < 4; ++j) (out + row_of(t, j) * p.dvp)[s_off] = w[t][j];
            }
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) u[t] = u[t] * tk[t];
        split8<3>(u[0], u[1], ub[0]);
        split8<3>(u[2], u[3], ub[1]);
        if (FWD && HALVES == 1) beside<18, 6>();
        // S = exp(c_63) S + K^T (exp(c_63 - c) u)
        KAN_FENCE();
        ahead(6);
#pragma unroll
        for (int g = 0; g < GROUP_N; ++g) {
            if (g == GROUP_N / 2) ahead(7);
            mma_tiles<2, PL, 3>(S + (g & ~1), kc[g % AHEAD], ub[g & 1]);
            KAN_FENCE();
            if (g + AHEAD < GROUP_N) load_cols<PL, DKP>(K, half * L::STEPS + (g + AHEAD) / 2, g & 1, kc[g % AHEAD]);
            KAN_FENCE();
        }
    }
    if constexpr (RUNS) {                              // [dkp][dvp + dkp]: B, then M
        float* const out = reinterpret_cast<float*>(ws + p.off_runs) + (seg * p.heads + bh) * DKP * (p.dvp + DKP) +
                           (of_m ? p.dvp : 0) + n0 + m;
        if (!of_m || n0 < DKP)
#pragma unroll
            for (int x = 0; x < DT; ++x)
#pragma unroll
                for (int j = 0; j < 4; ++j) out[(row_of(x0 + x, 4 * gq) + j) * (p.dvp + DKP)] = S[x][j];
    }
    if (!FWD) return;
    if (first < chunks) {
        __syncthreads();
        put_rows(chunks - 1);
    }
    // rows of this segment behind the sequence's end
    const int64_t past = len > (int64_t)first * C ? len : (int64_t)first * C;
    const int64_t last_row = seg + 1 < p.segs ? (int64_t)(first + p.seg_chunks) * C : d.T;
    for (int64_t e = lane + 64 * half; e < (last_row - past) * 16; e += 64 * HALVES) {
        const int64_t t = past + e / 16;
        const int nn = n0 + (int)(e % 16);
        if (nn < Dv) put(static_cast<TS*>(a.y) + ((b * d.T + t) * d.Hv + h) * Dv + nn, 0.0f);
    }
    // the last state is that of the segment with the sequence's end
    if (!a.hT || !mine || all > first + p.seg_chunks || (all <= first && seg > 0)) return;
#pragma unroll
    for (int x = 0; x < DT; ++x)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int dd = row_of(x0 + x, 4 * gq) + j;
            if (dd < Dk) a.hT[(bh * Dk + dd) * Dv + n0 + m] = S[x][j];
        }
}

// Backwards along a sequence: r, dv and the gradients of the chunks' last states.
// In segments the gradient of the state goes through one as M^T dS + F; RUNS finds
// F, what becomes of no gradient.
template <typename TS, int DKP, int GROUPS, bool EVEN, bool RUNS>
__global__ void __launch_bounds__((Scan<TS, DKP, GROUPS, kBack, EVEN>::NT))
    delta_back_kernel(kan_delta_desc_t d, DeltaPlan p, DeltaArgs a, char* ws) {
    typedef Scan<TS, DKP, GROUPS, kBack, EVEN> L;
    extern __shared__ __align__(16) char lds[];
    constexpr bool DIRECT = L::DIRECT;
    constexpr int PL = L::PL, NT = L::NT, W = L::W, DT = L::DT, HALVES = L::HALVES;
    int head, tile;
    head_and_tile((int)p.heads * p.segs, (int)((d.Dv + W - 1) / W), head, tile);
    const int seg = head / (int)p.heads;
    if (RUNS && seg == 0) return;                      // nothing comes before it
    const int64_t bh = head % (int)p.heads, b = bh / d.Hv, h = bh % d.Hv, hk = h / (d.Hv / d.Hk);
    const int tid = threadIdx.x, lane = tid & 63, m = lane & 15, gq = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), half = wave % HALVES, group = wave / HALVES;
    const int nb = tile * W, n0 = nb + 16 * group;
    const int Dk = (int)d.Dk, Dv = (int)d.Dv, len = length_of(a, b, d.T), all = (len + C - 1) / C;
    const int first = seg * p.seg_chunks, chunks = all < first + p.seg_chunks ? all : first + p.seg_chunks;
    const bool mine = n0 + m < Dv;
    const int x0 = half * DT;
    if (!RUNS) {                                       // rows of this segment behind the sequence's end
        const int64_t past = len > (int64_t)first * C ? len : (int64_t)first * C;
        const int64_t last_row = seg + 1 < p.segs ? (int64_t)(first + p.seg_chunks) * C : d.T;
        for (int64_t e = lane + 64 * half; e < (last_row - past) * 16; e += 64 * HALVES) {
            const int64_t t = past + e / 16;
            const int nn = n0 + (int)(e % 16);
            if (nn < Dv) put(static_cast<TS*>(a.dv) + at_row(d.dv, b, t, h) + nn, 0.0f);
        }
    }
    const float* start = a.dhT ? a.dhT + bh * Dk * Dv : nullptr;       // [Dk][Dv], or of the workspace [dkp][dvp]
    int start_row = Dv;
    if (RUNS) {
        start = nullptr;
    } else if (seg + 1 < p.segs) {
        start = reinterpret_cast<const float*>(ws + p.off_ends) + (seg * p.heads + bh) * DKP * p.dvp;
        start_row = p.dvp;
    }
    f32x4 S[DT];
#pragma unroll
    for (int x = 0; x < DT; ++x)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int dd = row_of(x0 + x, 4 * gq) + j;
            S[x][j] = start && dd < Dk && mine ? start[(int64_t)dd * start_row + n0 + m] : 0.0f;
        }
    const TS* const k_base = static_cast<const TS*>(a.k) + at_row(d.k, b, 0, hk);
    const TS* const q_base = static_cast<const TS*>(a.q) + at_row(d.q, b, 0, hk);
    const TS* const y_base = static_cast<const TS*>(a.dy) + (b * d.T * d.Hv + h) * Dv + nb;
    const float* const rows_base = reinterpret_cast<const float*>(ws + p.off_rows) + bh * p.chunks * kFields * C;
    const char* const mats_base = ws + p.off_mats + bh * p.chunks * p.mats + 3 * kTri * 2;     // G^T, P^T
    Carry<TS, DKP, NT, EVEN> ck, cq;
    Carry<TS, W, NT, EVEN> cy;
    CarryBytes<L::MATS * 2, NT> cm;
    CarryBytes<kFields * C * 4, NT> cr;
    Direct<DKP, NT> xk, xq;
    Direct<W, NT> xy;
    if (DIRECT) {
        xk.plan(d.k.row, Dk);
        xq.plan(d.q.row, Dk);
        xy.plan(d.Hv * Dv, Dv - nb);
    }
    const uint32_t s_off = 8 * gq * (uint32_t)p.dvp + n0 + m, v_row = (uint32_t)d.dv.row;
    const uint32_t v_off = 8 * gq * v_row + (mine ? n0 + m : 0);
    constexpr int PARTS = DIRECT ? 1 : 8;
    auto fetch = [&](int part, int n) {                // as in the scan above
        const int64_t t0 = (int64_t)n * C;
        const int rows = len - n * C;
        char* const to = lds + (DIRECT ? (n & 1) * L::BUF : 0);
        const char* const mats = mats_base + n * p.mats;
        const float* const fields = rows_base + (int64_t)n * kFields * C;
        constexpr int NK = ck.N, NY = cy.N, NM = cm.N, NF = cr.N, ALL = 2 * NK + NY + NM + NF;
#pragma unroll
        for (int j = 0; j < ALL; ++j) {
            if (j * PARTS / ALL != part) continue;
            const int q = j - NK, v = q - NK, x = v - NY, f = x - NM;
            if (j < NK) {
                if constexpr (DIRECT) xk.load(j, k_base + t0 * d.k.row, rows, to + L::K);
                else ck.load(j, k_base + t0 * d.k.row, d.k.row, rows, Dk);
            } else if (q < NK) {
                if constexpr (DIRECT) xq.load(q, q_base + t0 * d.q.row, rows, to + L::Q);
                else cq.load(q, q_base + t0 * d.q.row, d.q.row, rows, Dk);
            } else if (v < NY) {
                if constexpr (DIRECT) xy.load(v, y_base + t0 * d.Hv * Dv, rows, to + L::V);
                else cy.load(v, y_base + t0 * d.Hv * Dv, d.Hv * Dv, rows, Dv - nb);
            } else if (x < NM) {
                if constexpr (L::MATS_DIRECT)
                    DirectBytes<L::MATS * 2, NT>::load(x, mats, lds + L::G + (n & 1) * L::G_BUF);
                else cm.load(x, mats);
            } else {
                if constexpr (DIRECT) DirectBytes<kFields * C * 4, NT>::load(f, fields, to + L::FIELDS);
                else cr.load(f, fields);
            }
        }
    };
    char* const my_slot = lds + L::SLOT0 + wave * L::SLOT;
    const char* const other_slot = lds + L::SLOT0 + (wave ^ 1) * L::SLOT;
    // r and dv of a chunk, stored in the next one's time
    f32x4 r[4], dv[4];
    auto put_rows = [&](int n) {
        const int rows = len - n * C;
        float* const out_r = reinterpret_cast<float*>(ws + p.off_r) + (bh * p.chunks + n) * C * p.dvp;
        TS* const out_v = static_cast<TS*>(a.dv) + at_row(d.dv, b, (int64_t)n * C, h);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            if (HALVES == 2 && t / 2 != half) continue;                // uniform
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                (out_r + row_of(t, j) * p.dvp)[s_off] = r[t][j];
                if (rows >= C ? mine : mine && row_of(t, j) + 8 * gq < rows)
                    put(out_v + (uint32_t)row_of(t, j) * v_row + v_off, dv[t][j]);
            }
        }
    };
    if (first < chunks) {
#pragma unroll
        for (int part = 0; part < PARTS; ++part) fetch(part, chunks - 1);
    }
    for (int n = chunks - 1; n >= first; --n) {
        const int64_t ch = bh * p.chunks + n, t0 = (int64_t)n * C;
        const int rows = len - n * C;
        char* const buf = lds + (DIRECT ? (n & 1) * L::BUF : 0);
        if (DIRECT) arrived();
        __syncthreads();
        if (!DIRECT) {
            ck.store(reinterpret_cast<uint16_t*>(lds + L::K), rows, Dk);
            cq.store(reinterpret_cast<uint16_t*>(lds + L::Q), rows, Dk);
            cy.store(reinterpret_cast<uint16_t*>(lds + L::V), rows, Dv - nb);
            cr.store(lds + L::FIELDS);
        }
        if constexpr (!L::MATS_DIRECT) cm.store(lds + L::G);
        if (!DIRECT) __syncthreads();
        auto ahead = [&](int part) {
            if (part < PARTS && (!DIRECT || n > first)) fetch(part, n > first ? n - 1 : n);
        };
        ahead(0);
        if (!RUNS && n + 1 < chunks) put_rows(n + 1);
        const uint16_t* const K = reinterpret_cast<const uint16_t*>(buf + L::K);       // [PL][64][DKP]
        const uint16_t* const Q = reinterpret_cast<const uint16_t*>(buf + L::Q);
        const uint16_t* const Y = reinterpret_cast<const uint16_t*>(buf + L::V);       // [PL][64][W]: dY
        const float* const row = reinterpret_cast<const float*>(buf + L::FIELDS);
        const uint16_t* const G = reinterpret_cast<const uint16_t*>(lds + L::G + (n & 1) * L::G_BUF);  // [3][kTri]: G^T
        const uint16_t* const P = L::P_LDS ? G + 3 * kTri : reinterpret_cast<const uint16_t*>(mats_base + n * p.mats) + 3 * kTri;
        if (!RUNS) {
            float* const out_S = reinterpret_cast<float*>(ws + p.off_dS) + ch * DKP * p.dvp;
#pragma unroll
            for (int x = 0; x < DT; ++x)
#pragma unroll
                for (int j = 0; j < 4; ++j) (out_S + row_of(x0 + x, j) * p.dvp)[s_off] = S[x][j];
        }
        f32x4 fk[4], beta[4], tk[4], fq[4];            // the rows' factors, on their way meanwhile
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            fk[t] = at_rows(row, kFk, t);
            beta[t] = at_rows(row, kBeta, t);
            tk[t] = at_rows(row, kTk, t);
            fq[t] = at_rows(row, kFq, t);
        }
        const float whole = whole_decay(row);
        f32x4 kd[4], py[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) kd[t] = py[t] = zero4();
        bf16x8 yb[2][PL];                              // dY in this wave's columns
        bf16x8 unused[L::STEPS][1];
        rows_by_state<L, DKP, 1>(K, half * L::STEPS, S, kd, unused, ahead, [&] {
            col_frag<PL, W>(Y, 0, 2 * group + ((m & 3) >> 1), m & 1, yb[0]);
            col_frag<PL, W>(Y, 1, 2 * group + ((m & 3) >> 1), m & 1, yb[1]);
        });
        ahead(3);
        if (HALVES == 2) give_tiles(my_slot, kd, 4);
        if (HALVES == 2 || !L::MATS_DIRECT) __syncthreads();           // G^T and P^T are there, and the partner's part
        {
            bf16x8 pa[4][3], pb[2][3];
            load_tri<3, true, true>(P, pa);
            load_tri<3, true, false>(P, pb);
            if (HALVES == 2) add_tiles(other_slot, kd, 4);
            mma_tiles<4, 3, PL>(py, pa, yb[1]);
            mma_tiles<2, 3, PL>(py, pb, yb[0]);
        }
        bf16x8 ga[4][3], gb[2][3];
        load_tri<3, true, true>(G, ga);
        load_tri<3, true, false>(G, gb);
        KAN_FENCE();
        ahead(4);
        f32x4 y[4];                                    // dY as floats
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int z = 0; z < PL; ++z) {
                uint32_t wd[4];
                __builtin_memcpy(wd, &yb[s][z], 16);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float v = __uint_as_float(j & 1 ? wd[j / 2] & 0xffff0000u : wd[j / 2] << 16);
                    y[2 * s + (j >> 2)][j & 3] = z ? y[2 * s + (j >> 2)][j & 3] + v : v;
                }
            }
        {
            f32x4 gu[4], bu[4];
            bf16x8 ub[2][3];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                r[t] = py[t] + tk[t] * kd[t];          // du
                bu[t] = beta[t] * r[t];
                gu[t] = zero4();
            }
            split8<3>(bu[2], bu[3], ub[1]);
            split8<3>(bu[0], bu[1], ub[0]);
            mma_tiles<4, 3, 3>(gu, ga, ub[1]);
            mma_tiles<2, 3, 3>(gu, gb, ub[0]);
#pragma unroll
            for (int t = 0; t < 4; ++t) r[t] = r[t] - gu[t];
        }
        // columns of K and Q in turn, two groups ahead
        constexpr int GROUP_N = 4 * L::STEPS, AHEAD = PL == 1 ? 4 : 2;
        bf16x8 kc[AHEAD][2][PL];
        auto load_group = [&](int g) {
            load_cols<PL, DKP>(g & 2 ? Q : K, half * L::STEPS + g / 4, g & 1, kc[g % AHEAD]);
        };
#pragma unroll
        for (int g = 0; g < AHEAD; ++g) load_group(g);
        KAN_FENCE();
        ahead(5);
        f32x4 v[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            dv[t] = beta[t] * r[t];
            // rows of exp(c) (scale Q^T dY - K^T dv)
            y[t] = y[t] * fq[t];
            v[t] = -dv[t] * fk[t];
        }
        bf16x8 ys[2][3], vs[2][3];
        split8<3>(v[0], v[1], vs[0]);
        split8<3>(v[2], v[3], vs[1]);
        split8<3>(y[0], y[1], ys[0]);
        split8<3>(y[2], y[3], ys[1]);
#pragma unroll
        for (int x = 0; x < DT; ++x) S[x] = whole * S[x];
        KAN_FENCE();
        ahead(6);
#pragma unroll
        for (int g = 0; g < GROUP_N; ++g) {            // two tiles of the state by K, then by Q
            if (g == GROUP_N / 2) ahead(7);
            mma_tiles<2, PL, 3>(S + 2 * (g / 4), kc[g % AHEAD], g & 2 ? ys[g & 1] : vs[g & 1]);
            KAN_FENCE();
            if (g + AHEAD < GROUP_N) load_group(g + AHEAD);
            KAN_FENCE();
        }
    }
    if constexpr (RUNS) {
        float* const out = reinterpret_cast<float*>(ws + p.off_ends) + (seg * p.heads + bh) * DKP * p.dvp + n0 + m;
#pragma unroll
        for (int x = 0; x < DT; ++x)
#pragma unroll
            for (int j = 0; j < 4; ++j) out[(row_of(x0 + x, 4 * gq) + j) * p.dvp] = S[x][j];
        return;
    }
    if (first < chunks) put_rows(first);
    if (!a.dh0 || !mine || seg > 0) return;
#pragma unroll
    for (int x = 0; x < DT; ++x)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int dd = row_of(x0 + x, 4 * gq) + j;
            if (dd < Dk) a.dh0[(bh * Dk + dd) * Dv + n0 + m] = S[x][j];
        }
}

// The segments' starts, forward: S_1 = B_0, S_{s + 1} = M_s S_s + B_s; or their ends,
// BACK, in the place of F_s: dS_s = dhT for the last one, dS_{s - 1} = M_s^T dS_s + F_s.
// A block has 16 columns of a head, a wave 16 rows of them; the state is in LDS, as
// the right operand of the next product.
template <int DKP, bool BACK>
__global__ void __launch_bounds__(4 * DKP) delta_link_kernel(kan_delta_desc_t d, DeltaPlan p, DeltaArgs a, char* ws) {
    constexpr int STEPS = DKP / 32;
    __shared__ __align__(16) uint16_t S[2][3][16][DKP + 8];
    const int64_t bh = blockIdx.x % (unsigned)p.heads;
    const int n0 = (int)(blockIdx.x / (unsigned)p.heads) * 16, Dk = (int)d.Dk, Dv = (int)d.Dv;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, m = lane & 15, gq = lane >> 4, row = 16 * wave + 4 * gq;
    const int64_t state = (int64_t)DKP * p.dvp, run = (int64_t)DKP * (p.dvp + DKP), at = (int64_t)row * p.dvp + n0 + m;
    const float* const runs = reinterpret_cast<const float*>(ws + p.off_runs);
    float* const ends = reinterpret_cast<float*>(ws + p.off_ends);
    float* const starts = reinterpret_cast<float*>(ws + p.off_starts);
    f32x4 v, next = zero4();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (BACK) v[j] = a.dhT && row + j < Dk && n0 + m < Dv ? a.dhT[(bh * Dk + row + j) * Dv + n0 + m] : 0.0f;
        else v[j] = runs[bh * run + (int64_t)(row + j) * (p.dvp + DKP) + n0 + m];
        if (BACK) next[j] = ends[((p.segs - 1) * p.heads + bh) * state + at + (int64_t)j * p.dvp];
    }
    for (int k = 1; k < p.segs; ++k) {
        // forward: v is the start of segment s = k; back: the end of segment s = segs - k, and next is F_s
        const int s = BACK ? p.segs - k : k;
        const float* const M = runs + (s * p.heads + bh) * run + p.dvp;
        if (!BACK) {
            float* const out = starts + (s * p.heads + bh) * state + at;
#pragma unroll
            for (int j = 0; j < 4; ++j) out[(int64_t)j * p.dvp] = v[j];
            if (k + 1 == p.segs) return;
            const float* const B = runs + (s * p.heads + bh) * run + (int64_t)row * (p.dvp + DKP) + n0 + m;
#pragma unroll
            for (int j = 0; j < 4; ++j) next[j] = B[(int64_t)j * (p.dvp + DKP)];
        }
        bf16x8 planes[3];
        split8<3>(v, zero4(), planes);
#pragma unroll
        for (int z = 0; z < 3; ++z) __builtin_memcpy(&S[k & 1][z][m][row], &planes[z], 8);
        __syncthreads();
#pragma unroll
        for (int q = 0; q < STEPS; ++q) {
            const int c = 32 * q + 8 * gq;
            f32x4 lo, hi;
            if (BACK) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    lo[j] = M[(int64_t)(c + j) * (p.dvp + DKP) + 16 * wave + m];
                    hi[j] = M[(int64_t)(c + 4 + j) * (p.dvp + DKP) + 16 * wave + m];
                }
            } else {
                lo = ld4(M + (int64_t)(16 * wave + m) * (p.dvp + DKP) + c);
                hi = ld4(M + (int64_t)(16 * wave + m) * (p.dvp + DKP) + c + 4);
            }
            bf16x8 ma[3], sb[3];
            split8<3>(lo, hi, ma);
#pragma unroll
            for (int z = 0; z < 3; ++z) sb[z] = *reinterpret_cast<const bf16x8*>(&S[k & 1][z][m][c]);
            mma<3, 3>(next, ma, sb);
        }
        v = next;
        if (BACK) {                                    // this lane's values of F_{s - 1} make room for dS_{s - 1}
            float* const out = ends + ((s - 1) * p.heads + bh) * state + at;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (s > 1) next[j] = out[(int64_t)j * p.dvp];
                out[(int64_t)j * p.dvp] = v[j];
            }
        }
    }
}

// ---- gradients of a chunk's rows -----------------------------------------------------

// A block has a chunk; wave w rows 16 w .. + 15, of which lane (gq, m) has row 16 w + m in
// four columns 16 x + 4 gq .. of every tile x.  The products with the states come
// first, 32 of their columns at a time through LDS, then those of the rows among
// themselves, in the same place: with bfloat16 rows two blocks fit a compute unit
// and hide each other's loads (4 x 4096 x 16 x 128 bf16: 479 us with one, 319 with two).
constexpr int GRAD_NT = 256, GS = 32;                // GS: state columns at a time
__device__ __forceinline__ int slice_at(int row, int c) { return row * GS + ((c ^ (row >> 2)) & 3) * 8; }
__device__ __forceinline__ float quad_sum(float v) {  // over the four lanes of a row
    v += __shfl_xor(v, 16, 64);
    return v + __shfl_xor(v, 32, 64);
}
template <typename TS>
__device__ __forceinline__ void put4(TS* p, int at, int D, const f32x4& v) {
    if (at + 4 <= D) {
        const float t[4] = {v[0], v[1], v[2], v[3]};
        store_vec<4>(p + at, t);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (at + j < D) put(p + at + j, v[j]);
    }
}
// Four values of a row in LDS planes, columns 16 x + 4 gq ..
template <int PL, int W>
__device__ __forceinline__ f32x4 row_values(const uint16_t* lds, int row, int x, int gq) {
    f32x4 v = zero4();
#pragma unroll
    for (int n = 0; n < PL; ++n) {
        uint32_t w[2];
        __builtin_memcpy(w, lds + n * C * W + piece_at<W>(row, 2 * x + (gq >> 1)) + 4 * (gq & 1), 8);
        const f32x4 t = {__uint_as_float(w[0] << 16), __uint_as_float(w[0] & 0xffff0000u), __uint_as_float(w[1] << 16),
                         __uint_as_float(w[1] & 0xffff0000u)};
        v = n ? v + t : t;
    }
    return v;
}

template <typename TS, int DKP>
constexpr int grad_bytes() {                           // of the states' slices, or of the rows and their pairs
    constexpr int states = 3 * GS * (2 * DKP + C) * 2, pairs = planes_of<TS>::n * C * 2 * DKP * 2 + 2 * C * LC * 4;
    return states > pairs ? states : pairs;
}
template <typename TS, int DKP>
__global__ void __launch_bounds__(GRAD_NT, sizeof(TS) == 2 ? 2 : 1) delta_grad_kernel(kan_delta_desc_t d, DeltaPlan p, DeltaArgs a, char* ws) {
    extern __shared__ __align__(16) char lds[];
    constexpr int PL = planes_of<TS>::n, DT = DKP / 16, NT = GRAD_NT;
    uint16_t* const S0 = reinterpret_cast<uint16_t*>(lds);         // [3][DKP][32]
    uint16_t* const S1 = S0 + 3 * DKP * GS;                        // [3][DKP][32]: dS
    uint16_t* const U = S1 + 3 * DKP * GS;                         // [3][64][32]: u
    uint16_t* const K = reinterpret_cast<uint16_t*>(lds);          // [PL][64][DKP], after the states
    uint16_t* const Q = K + PL * C * DKP;
    float* const PD = reinterpret_cast<float*>(Q + PL * C * DKP);  // [64][LC]: scale dP D; then dP P - X A
    float* const XD = PD + C * LC;                                 // X D
    float* const row = reinterpret_cast<float*>(lds + grad_bytes<TS, DKP>());
    float* const xs = row + kFields * C;                           // [64] parts of rows that come from S0
    float* const zs = xs + C;                                      // [64] parts of rows that reach dS1
    float* const sums = zs + C;                                    // [4][64] parts of dg
    float* const part = sums + 4 * C;                              // [4] of <dS1, S0>
    const int64_t n = blockIdx.x % (unsigned)p.chunks, bh = blockIdx.x / (unsigned)p.chunks;
    const int64_t b = bh / d.Hv, h = bh % d.Hv, share = d.Hv / d.Hk, hk = h / share;
    const int64_t t0 = n * C, ch = bh * p.chunks + n;
    const int Dk = (int)d.Dk, Dv = (int)d.Dv;
    const int rows = length_of(a, b, d.T) - (int)t0;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, m = lane & 15, gq = lane >> 4;
    const int inside = (int)(d.T - t0 < C ? d.T - t0 : C);         // rows of the chunk that the arrays have
    const int im = 16 * wave + m;                                  // this lane's row
    TS* const dq = static_cast<TS*>(a.dq) + at_row(d.dq, b, t0 + im, hk);
    TS* const dk = static_cast<TS*>(a.dk) + at_row(d.dk, b, t0 + im, hk);
    if (rows <= 0) {                                               // uniform
        if (tid < inside) {
            a.dg[(b * d.T + t0 + tid) * d.Hv + h] = 0.0f;
            a.dbeta[(b * d.T + t0 + tid) * d.Hv + h] = 0.0f;
        }
        if (share == 1 && im < inside)
#pragma unroll
            for (int x = 0; x < DT; ++x) {
                put4(dq, 16 * x + 4 * gq, Dk, zero4());
                put4(dk, 16 * x + 4 * gq, Dk, zero4());
            }
        return;
    }
    {
        CarryBytes<kFields * C * 4, NT> cr;
        cr.load(reinterpret_cast<const float*>(ws + p.off_rows) + ch * kFields * C);
        cr.store(row);
    }
    const float* const in_S = reinterpret_cast<const float*>(ws + p.off_S) + ch * DKP * p.dvp;
    const float* const in_dS = reinterpret_cast<const float*>(ws + p.off_dS) + ch * DKP * p.dvp;
    const float* const in_w = reinterpret_cast<const float*>(ws + p.off_w) + (ch * C + im) * p.dvp;
    const float* const in_r = reinterpret_cast<const float*>(ws + p.off_r) + (ch * C + im) * p.dvp;
    const TS* const dy = static_cast<const TS*>(a.dy) + ((b * d.T + t0 + (im < rows ? im : 0)) * d.Hv + h) * Dv;
    const float* const rows_at = reinterpret_cast<const float*>(ws + p.off_rows) + ch * kFields * C;
    const float beta_m = rows_at[kBeta * C + im];
    f32x4 ys[DT], vs[DT], us[DT], dP[4], X[4];
#pragma unroll
    for (int x = 0; x < DT; ++x) ys[x] = vs[x] = us[x] = zero4();
#pragma unroll
    for (int x = 0; x < 4; ++x) dP[x] = X[x] = zero4();
    float rw = 0.0f, ss = 0.0f;
    constexpr int SP = DKP * GS / 8 / NT > 0 ? DKP * GS / 8 / NT : 1;      // pieces of a state's slice, a thread
    Piece<float> s0[SP], s1[SP];
    Piece<TS> py;
    f32x4 wn[2], rn[2];
    auto fetch = [&](int s) {
#pragma unroll
        for (int x = 0; x < SP; ++x) {
            const int e = tid + NT * x, dd = e / (GS / 8), c = e % (GS / 8);
            if (e >= DKP * GS / 8) break;
            load_piece(s0[x], in_S + dd * p.dvp + GS * s, 8 * c, GS);
            load_piece(s1[x], in_dS + dd * p.dvp + GS * s, 8 * c, GS);
        }
        const int at = GS * s + 8 * gq;
        if (im < rows && at < Dv) load_piece(py, dy, at, Dv);
        else no_piece(py);
#pragma unroll
        for (int z = 0; z < 2; ++z) wn[z] = ld4(in_w + at + 4 * z), rn[z] = ld4(in_r + at + 4 * z);
    };
    const int steps = (Dv + GS - 1) / GS;
    for (int s = 0; s < steps; ++s) {
        fetch(s);
        bf16x8 ya[PL], ua[3], va[3];
        piece_planes(py, ya);
#pragma unroll
        for (int z = 0; z < 2; ++z)
#pragma unroll
            for (int j = 0; j < 4; ++j) rw = __builtin_fmaf(wn[z][j], rn[z][j], rw);
        split8<3>(beta_m * wn[0], beta_m * wn[1], ua);
        split8<3>(beta_m * rn[0], beta_m * rn[1], va);
        __syncthreads();                               // the slice before is done with LDS
#pragma unroll
        for (int x = 0; x < SP; ++x) {
            const int e = tid + NT * x, dd = e / (GS / 8), c = e % (GS / 8);
            if (e >= DKP * GS / 8) break;
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = __builtin_fmaf(s0[x].v[j], s1[x].v[j], ss);
            bf16x8 v[3];
            piece_planes(s0[x], v);
#pragma unroll
            for (int z = 0; z < 3; ++z) *reinterpret_cast<bf16x8*>(S0 + z * DKP * GS + slice_at(dd, c)) = v[z];
            piece_planes(s1[x], v);
#pragma unroll
            for (int z = 0; z < 3; ++z) *reinterpret_cast<bf16x8*>(S1 + z * DKP * GS + slice_at(dd, c)) = v[z];
        }
#pragma unroll
        for (int z = 0; z < 3; ++z) *reinterpret_cast<bf16x8*>(U + z * C * GS + slice_at(im, gq)) = ua[z];
        __syncthreads();
#pragma unroll
        for (int x = 0; x < DT; ++x) {
            bf16x8 sb[3], db[3];
#pragma unroll
            for (int z = 0; z < 3; ++z) {
                sb[z] = *reinterpret_cast<const bf16x8*>(S0 + z * DKP * GS + slice_at(16 * x + m, gq));
                db[z] = *reinterpret_cast<const bf16x8*>(S1 + z * DKP * GS + slice_at(16 * x + m, gq));
            }
            mma<3, PL>(ys[x], sb, ya);
            mma<3, 3>(vs[x], sb, va);
            mma<3, 3>(us[x], db, ua);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            if (x > wave) break;
            bf16x8 ub[3];
#pragma unroll
            for (int z = 0; z < 3; ++z) ub[z] = *reinterpret_cast<const bf16x8*>(U + z * C * GS + slice_at(16 * x + m, gq));
            mma<3, PL>(dP[x], ub, ya);
            mma<3, 3>(X[x], ub, va);
        }
    }
    rw = quad_sum(rw);
    if (gq == 0 && im < inside) a.dbeta[(b * d.T + t0 + im) * d.Hv + h] = im < rows ? rw : 0.0f;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) ss += __shfl_xor(ss, o, 64);
    if (lane == 0) part[wave] = ss;
    __syncthreads();                                   // the states' slices are done with
    {
        Carry<TS, DKP, NT, false> ck, cq;
        ck.load(static_cast<const TS*>(a.k) + at_row(d.k, b, t0, hk), d.k.row, rows, Dk);
        cq.load(static_cast<const TS*>(a.q) + at_row(d.q, b, t0, hk), d.q.row, rows, Dk);
        ck.store(K, rows, Dk);
        cq.store(Q, rows, Dk);
    }
    __syncthreads();
    // the states' parts, with their factors; gradients of q and k as they were divided
    const float from = __builtin_amdgcn_exp2f(row[kHi * C + im] + row[kLo * C + im]), to = decay(row, C - 1, im);
    const float nk = row[kNk * C + im], nq = row[kNq * C + im];
    float xr = 0.0f, zr = 0.0f;
#pragma unroll
    for (int x = 0; x < DT; ++x) {
        const f32x4 qv = nq * row_values<PL, DKP>(Q, im, x, gq), kv = nk * row_values<PL, DKP>(K, im, x, gq);
        ys[x] = (d.scale * from) * ys[x];
        vs[x] = from * vs[x];
        us[x] = to * us[x];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            xr += qv[j] * ys[x][j] - kv[j] * vs[x][j];
            zr += kv[j] * us[x][j];
        }
        us[x] = us[x] - vs[x];                         // dk so far; ys: dq so far
    }
    xr = quad_sum(xr);
    zr = quad_sum(zr);
    if (gq == 0) xs[im] = xr, zs[im] = zr;
    // pairs of rows: this lane's row i = im against rows j = 16 x + 4 gq ..
    f32x4 qk[4], kk[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) qk[x] = kk[x] = zero4();
#pragma unroll
    for (int s = 0; s < DKP / 32; ++s) {
        bf16x8 ka[PL], qa[PL];
        row_frag<PL, DKP>(K, im, 4 * s + gq, ka);
        row_frag<PL, DKP>(Q, im, 4 * s + gq, qa);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            if (x > wave) break;
            bf16x8 kb[PL];
            row_frag<PL, DKP>(K, 16 * x + m, 4 * s + gq, kb);
            mma<PL, PL>(qk[x], kb, qa);
            mma<PL, PL>(kk[x], kb, ka);
        }
    }
    f32x4 e[4];                                        // dP P - X A
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        const int j0 = 16 * x + 4 * gq;
        const f32x4 nj = ld4(row + kNk * C + j0);
        f32x4 pd, xd;
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            const int j = j0 + y;
            const float D = j <= im ? decay(row, im, j) : 0.0f;
            pd[y] = j <= im ? d.scale * (dP[x][y] * D) : 0.0f;
            xd[y] = j < im ? X[x][y] * D : 0.0f;
            e[x][y] = j < im ? nj[y] * (pd[y] * (nq * qk[x][y]) - xd[y] * (nk * kk[x][y])) : 0.0f;
        }
        st4(PD + im * LC + j0, pd);
        st4(XD + im * LC + j0, xd);
    }
    __syncthreads();
    // products of the pairs with the rows, which are divided here by their pair's factor
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const int j0 = 32 * s + 8 * gq;
        f32x4 pr[2], pc[2], xc[2];
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            const f32x4 nkj = ld4(row + kNk * C + j0 + 4 * z), nqj = ld4(row + kNq * C + j0 + 4 * z);
            pr[z] = ld4(PD + im * LC + j0 + 4 * z) * nkj;
            xc[z] = ld4(XD + im * LC + j0 + 4 * z);
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int j = j0 + 4 * z + y;
                pc[z][y] = PD[j * LC + im];
                xc[z][y] += XD[j * LC + im];
            }
            pc[z] = pc[z] * nqj;
            xc[z] = -xc[z] * nkj;
        }
        bf16x8 pra[3], pca[3], xca[3];
        split8<3>(pr[0], pr[1], pra);
        split8<3>(pc[0], pc[1], pca);
        split8<3>(xc[0], xc[1], xca);
#pragma unroll
        for (int x = 0; x < DT; ++x) {
            bf16x8 kt[PL], qt[PL];
            col_frag<PL, DKP>(K, s, 2 * x + ((m & 3) >> 1), m & 1, kt);
            if (s <= wave / 2) mma<PL, 3>(ys[x], kt, pra);
            if (s >= wave / 2) {
                col_frag<PL, DKP>(Q, s, 2 * x + ((m & 3) >> 1), m & 1, qt);
                mma<PL, 3>(us[x], qt, pca);
            }
            mma<PL, 3>(us[x], kt, xca);
        }
    }
    // dg of row t, a lane each: pairs i >= t > j, of which a wave has 16 rows i, ...
    __syncthreads();
#pragma unroll
    for (int x = 0; x < 4; ++x) st4(PD + im * LC + 16 * x + 4 * gq, e[x]);     // this wave's rows
    float dg = 0.0f;
#pragma unroll
    for (int y = 0; y < 16; ++y) {
        const int i = 16 * wave + y;
        float sum = PD[i * LC + lane];
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const float before = __shfl_up(sum, o, 64);
            if (lane >= o) sum += before;
        }
        const float before = __shfl_up(sum, 1, 64);    // columns j < t
        if (i >= lane && lane > 0) dg += before;
    }
    sums[wave * C + lane] = dg;
    __syncthreads();
    // ... rows i >= t that start from S0, rows j < t that reach dS1, and the state itself
    if (wave == 0) {
        float x = xs[lane], z = zs[lane];
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const float after = __shfl_down(x, o, 64), before = __shfl_up(z, o, 64);
            if (lane + o < 64) x += after;
            if (lane >= o) z += before;
        }
        const float earlier = __shfl_up(z, 1, 64);
        dg = ((sums[lane] + sums[C + lane]) + (sums[2 * C + lane] + sums[3 * C + lane])) + x + (lane > 0 ? earlier : 0.0f) +
             whole_decay(row) * (part[0] + part[1] + part[2] + part[3]);
        if (lane < inside) a.dg[(b * d.T + t0 + lane) * d.Hv + h] = lane < rows ? dg : 0.0f;
    }
    if (im >= inside) return;
    if (share > 1) {
        if (im >= rows) return;
        const int64_t at = ((b * d.T + t0 + im) * d.Hv + h) * Dk;
#pragma unroll
        for (int x = 0; x < DT; ++x) {
            put4(reinterpret_cast<float*>(ws + p.off_dq) + at, 16 * x + 4 * gq, Dk, ys[x]);
            put4(reinterpret_cast<float*>(ws + p.off_dk) + at, 16 * x + 4 * gq, Dk, us[x]);
        }
        return;
    }
    if (d.flags & KAN_DELTA_UNIT) {                    // through x / sqrt(x.x + eps)
        float qd = 0.0f, kd = 0.0f;
#pragma unroll
        for (int x = 0; x < DT; ++x) {
            const f32x4 qv = row_values<PL, DKP>(Q, im, x, gq), kv = row_values<PL, DKP>(K, im, x, gq);
#pragma unroll
            for (int j = 0; j < 4; ++j) qd += qv[j] * ys[x][j], kd += kv[j] * us[x][j];
        }
        qd = quad_sum(qd) * nq * nq;
        kd = quad_sum(kd) * nk * nk;
#pragma unroll
        for (int x = 0; x < DT; ++x) {
            const f32x4 qv = row_values<PL, DKP>(Q, im, x, gq), kv = row_values<PL, DKP>(K, im, x, gq);
            ys[x] = nq * (ys[x] - qd * qv);
            us[x] = nk * (us[x] - kd * kv);
        }
    }
#pragma unroll
    for (int x = 0; x < DT; ++x) {
        put4(dq, 16 * x + 4 * gq, Dk, im < rows ? ys[x] : zero4());
        put4(dk, 16 * x + 4 * gq, Dk, im < rows ? us[x] : zero4());
    }
}

constexpr int NT = 256;              // threads of the row-wise kernels' blocks
template <typename TS>
__device__ __forceinline__ f32x4 row4(const TS* p, int at, int D) {    // zero past the row's end
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
    __shared__ float ks[kDeltaMaxDk], qs[kDeltaMaxDk], red[2][16][68];
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
    const float alpha = expf(a.g[b * d.Hv + h]), beta = a.beta[b * d.Hv + h];
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

template <typename K, typename... Args>
hipError_t launch(K kernel, int64_t blocks, int threads, size_t lds, hipStream_t s, Args... args) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3((unsigned)threads), lds, s, args...);
    return hipGetLastError();
}

template <typename TS, int DKP, bool BWD>
hipError_t prep(const kan_delta_desc_t& d, const DeltaPlan& p, const DeltaArgs& a, char* ws, hipStream_t s) {
    constexpr size_t lds = prep_bytes<TS, DKP>() + 4 * kFields * C;
    const int64_t blocks = d.B * d.Hk * p.chunks;
    return d.Hv > d.Hk ? launch(delta_prep_kernel<TS, DKP, BWD, true>, blocks, PREP_NT, lds, s, d, p, a, ws)
                       : launch(delta_prep_kernel<TS, DKP, BWD, false>, blocks, PREP_NT, lds, s, d, p, a, ws);
}
template <typename TS, int DKP, int GROUPS, int PASS, bool EVEN>
hipError_t scan_e(const kan_delta_desc_t& d, const DeltaPlan& p, const DeltaArgs& a, char* ws, bool runs,
                  hipStream_t s) {
    typedef Scan<TS, DKP, GROUPS, PASS, EVEN> L;
    static_assert(L::LDS <= 160 * 1024, "LDS of a compute unit");
    const int64_t tiles = (d.Dv + L::W - 1) / L::W + (PASS == kRuns ? (DKP + L::W - 1) / L::W : 0);
    const int64_t blocks = p.heads * (PASS == kRuns ? p.runs : p.segs) * tiles;
    if constexpr (PASS == kBack) {
        if (runs) return launch(delta_back_kernel<TS, DKP, GROUPS, EVEN, true>, blocks, L::NT, L::LDS, s, d, p, a, ws);
        return launch(delta_back_kernel<TS, DKP, GROUPS, EVEN, false>, blocks, L::NT, L::LDS, s, d, p, a, ws);
    } else {
        return launch(delta_scan_kernel<TS, DKP, GROUPS, PASS, EVEN>, blocks, L::NT, L::LDS, s, d, p, a, ws);
    }
}
template <int DKP, bool BACK>
hipError_t link(const kan_delta_desc_t& d, const DeltaPlan& p, const DeltaArgs& a, char* ws, hipStream_t s) {
    return launch(delta_link_kernel<DKP, BACK>, p.heads * ((d.Dv + 15) / 16), 4 * DKP, 0, s, d, p, a, ws);
}
template <typename TS, int DKP, int PASS>
hipError_t scan(const kan_delta_desc_t& d, const DeltaPlan& p, const DeltaArgs& a, char* ws, hipStream_t s,
                bool runs = false) {
    // pieces of eight, on 16 bytes where they go to LDS directly
    auto direct = [](const void* at, const kan_heads_t& s) {
        return aligned(at, 16) && s.seq % 8 == 0 && s.row % 8 == 0 && s.head % 8 == 0;
    };
    bool even = d.Dk % 8 == 0 && d.Dv % 8 == 0;
    if (sizeof(TS) == 2)
        even = even && direct(a.k, d.k) && (PASS == kStates || PASS == kRuns || direct(a.q, d.q)) &&
               (PASS == kBack || direct(a.v, d.v));
    constexpr int WIDE = sizeof(TS) == 4 && PASS == kBack ? 2 : 4;     // groups of 16 columns that LDS has room for
    // cut sequences have too few heads for wide blocks
    if constexpr (WIDE == 4 && PASS != kRuns)
        if (p.groups == 4)
            return even ? scan_e<TS, DKP, 4, PASS, true>(d, p, a, ws, runs, s) : scan_e<TS, DKP, 4, PASS, false>(d, p, a, ws, runs, s);
    return even ? scan_e<TS, DKP, 2, PASS, true>(d, p, a, ws, runs, s) : scan_e<TS, DKP, 2, PASS, false>(d, p, a, ws, runs, s);
}
template <typename TS, int DKP>
hipError_t grad(const kan_delta_desc_t& d, const DeltaPlan& p, const DeltaArgs& a, char* ws, hipStream_t s) {
    constexpr size_t lds = grad_bytes<TS, DKP>() + 4 * kFields * C + 24 * C + 16;
    return launch(delta_grad_kernel<TS, DKP>, p.heads * p.chunks, GRAD_NT, lds, s, d, p, a, ws);
}
// The segments' starts, where sequences are cut.
template <typename TS, int DKP>
hipError_t starts(const kan_delta_desc_t& d, const DeltaPlan& p, const DeltaArgs& a, char* ws, hipStream_t s) {
    if (p.segs == 1) return hipSuccess;
    const hipError_t e = scan<TS, DKP, kRuns>(d, p, a, ws, s);
    return e != hipSuccess ? e : link<DKP, false>(d, p, a, ws, s);
}
template <typename TS, int DKP>
hipError_t forward(const kan_delta_desc_t& d, const DeltaPlan& p, const DeltaArgs& a, char* ws, hipStream_t s) {
    hipError_t e = hipSuccess;
    if (p.chunks > 0) e = prep<TS, DKP, false>(d, p, a, ws, s);
    if (e == hipSuccess) e = starts<TS, DKP>(d, p, a, ws, s);
    return e != hipSuccess ? e : scan<TS, DKP, kForward>(d, p, a, ws, s);
}
template <typename TS, int DKP>
hipError_t backward(const kan_delta_desc_t& d, const DeltaPlan& p, const DeltaArgs& a, char* ws, hipStream_t s) {
    hipError_t e = hipSuccess;
    if (p.chunks > 0) {
        e = prep<TS, DKP, true>(d, p, a, ws, s);
        if (e == hipSuccess) e = starts<TS, DKP>(d, p, a, ws, s);
        if (e == hipSuccess) e = scan<TS, DKP, kStates>(d, p, a, ws, s);
        if (e == hipSuccess && p.segs > 1) e = scan<TS, DKP, kBack>(d, p, a, ws, s, true);
        if (e == hipSuccess && p.segs > 1) e = link<DKP, true>(d, p, a, ws, s);
    }
    if (e == hipSuccess) e = scan<TS, DKP, kBack>(d, p, a, ws, s);
    if (e != hipSuccess || p.chunks == 0) return e;
    if ((e = grad<TS, DKP>(d, p, a, ws, s)) != hipSuccess || d.Hv == d.Hk) return e;
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
