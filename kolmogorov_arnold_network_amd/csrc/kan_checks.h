// Argument checks shared by the entry points of the operators over tokens.
#pragma once

#include "kan_internal.h"

namespace kan {

inline bool dtype_ok(int dtype) { return dtype == KAN_F32 || dtype == KAN_BF16; }
inline bool index_ok(int t) { return t == KAN_I32 || t == KAN_I64; }
inline bool size_ok(int64_t n, int64_t least) { return n >= least && n <= kIndexLimit; }
inline size_t index_bytes(int t) { return t == KAN_I32 ? 4 : 8; }

// Outputs against inputs and against each other.
template <int NO, int NI>
bool any_overlap(const Range (&outs)[NO], const Range (&ins)[NI]) {
    for (int a = 0; a < NO; ++a) {
        for (int b = 0; b < NI; ++b)
            if (overlap(outs[a], ins[b])) return true;
        for (int b = a + 1; b < NO; ++b)
            if (overlap(outs[a], outs[b])) return true;
    }
    return false;
}

template <int NP>
bool all_aligned(const void* const (&ptrs)[NP], uintptr_t a) {
    for (const void* p : ptrs)
        if (p && !aligned(p, a)) return false;
    return true;
}

inline int check_ws(const void* ws, size_t bytes, size_t need) {
    if (bytes < need) return KAN_ERR_WORKSPACE;
    if (need > 0 && !ws) return KAN_ERR_NULL;
    return ws && !aligned(ws, 256) ? KAN_ERR_ALIGN : KAN_OK;
}

// Strided rows [B][T][D].  A stride past 2^40 elements is refused, so that
// extents fit 64 bits with any B and T.
constexpr int64_t kStrideLimit = int64_t(1) << 40;
inline bool stride_ok(int64_t s) { return s >= 0 && s <= kStrideLimit; }
// Elements from the first to the last of the array, or -1 past 2^60.
inline int64_t extent(int64_t B, int64_t T, int64_t D, int64_t row, int64_t seq) {
    if (B == 0 || T == 0) return 0;
    const __int128 n = (__int128)(B - 1) * seq + (__int128)(T - 1) * row + D;
    return n > ((__int128)1 << 60) ? -1 : (int64_t)n;
}
// The least distance between the starts of two rows: 0 where rows of the
// array may interleave in another way than one stride inside the other.
inline int64_t row_distance(int64_t B, int64_t T, int64_t row, int64_t seq) {
    if (B <= 1 && T <= 1) return INT64_MAX;
    if (B <= 1) return row;
    if (T <= 1) return seq;
    const __int128 in_rows = (__int128)seq - (__int128)(T - 1) * row;   // sequences apart
    const __int128 in_seqs = (__int128)row - (__int128)(B - 1) * seq;   // sequences interleaved
    if (in_rows > 0) return (int64_t)std::min<__int128>(row, in_rows);
    if (in_seqs > 0) return (int64_t)std::min<__int128>(seq, in_seqs);
    return 0;
}

}  // namespace kan
