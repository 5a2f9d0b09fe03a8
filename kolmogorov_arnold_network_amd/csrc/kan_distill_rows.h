// How a row of the distillation kernels is dealt to parts and threads; host and
// device.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kan {

// A row is a head of single elements up to the first cache line of what is
// written (of z, where nothing is), vectors, and a tail of fewer elements than
// a vector.  Rows of an odd length start anywhere; lines cut between lanes and
// waves cost 20% of a step with 50021 bf16 logits (241 us against 204 at 50024).
// Thread i takes element i of the head and of the tail.
template <typename T>
__host__ __device__ inline int head_of(const T* p, int64_t V) {
    const int n = (int)((128 - (reinterpret_cast<uintptr_t>(p) & 127)) & 127) / (int)sizeof(T);
    return n < V ? n : (int)V;
}

// Part p of a row that is cut for several blocks: elements [v0, v1), the first
// part with the head, vectors from v, and the part that ends the row with the
// tail, `tail` on.  Parts are `part` elements of vectors; with a head the last
// one may be empty (v0 = v1).
struct Part {
    int64_t v0, v1, v, tail;
    __host__ __device__ inline Part(int p, int64_t part, int head, int64_t V, int VE) {
        v = head + p * part;
        v0 = !p ? 0 : v < V ? v : V;
        v1 = v + part < V ? v + part : V;
        tail = v0 < V && v1 == V ? V - (V - head) % VE : V;
    }
};

// The thread that stores element v of a row: vectors of VE go to the threads in
// turn, from the head on, and a part is a whole number of turns.
__host__ __device__ inline int owner_of(int64_t v, int head, int64_t V, int VE, int threads) {
    if (v < head) return (int)v;
    const int64_t tail = V - (V - head) % VE;
    return v < tail ? (int)((uint32_t)(v - head) / (uint32_t)VE % (uint32_t)threads) : (int)(v - tail);
}

}  // namespace kan
