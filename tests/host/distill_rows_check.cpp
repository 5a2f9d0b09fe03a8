// Host check of how the distillation kernels deal a row to threads
// (kan_distill_rows.h): walks the kernels' store loops for rows of all starts
// within a cache line and lengths around a whole number of vectors, turns and
// parts, and checks that every element is stored by one thread of one block,
// and that this is the thread that owner_of names, which stores a teacher's
// entry over it.  Exit status 0 and "ok <elements>": everything held.
#include <stdio.h>
#include <stdlib.h>

#include <initializer_list>
#include <vector>

#include "kan_distill_rows.h"

using namespace kan;

static long elements = 0;

static void need(bool ok, const char* what, int64_t V, int start, int VE, int threads, int64_t v) {
    if (ok) return;
    fprintf(stderr, "%s: V %lld, start %d, vectors of %d, %d threads, element %lld\n", what, (long long)V, start, VE,
            threads, (long long)v);
    exit(1);
}

// A row of V elements of `bytes` that starts `start` elements past a line, in `parts` parts of `part`.
static void walk(int64_t V, int start, int bytes, int VE, int threads, int parts, int64_t part) {
    const char* at = reinterpret_cast<const char*>(uintptr_t(4096)) + start * bytes;
    const int head = bytes == 4 ? head_of(reinterpret_cast<const float*>(at), V)
                                : head_of(reinterpret_cast<const uint16_t*>(at), V);
    std::vector<int> block(V, -1), thread(V, -1);
    auto store = [&](int b, int t, int64_t v) {
        need(v >= 0 && v < V, "outside the row", V, start, VE, threads, v);
        need(block[v] < 0, "stored twice", V, start, VE, threads, v);
        block[v] = b, thread[v] = t;
    };
    const int64_t stride = (int64_t)threads * VE;
    for (int p = 0; p < parts; ++p) {
        const Part r(p, part, head, V, VE);
        for (int t = 0; t < threads; ++t) {
            for (int64_t v = r.v + (int64_t)t * VE; v + VE <= r.v1; v += stride)
                for (int i = 0; i < VE; ++i) store(p, t, v + i);
            if (p == 0 && t < head) store(p, t, t);
            if (r.tail + t < V) store(p, t, r.tail + t);
        }
        for (int64_t v = r.v0; v < r.v1; ++v) need(block[v] == p, "not of its part", V, start, VE, threads, v);
    }
    for (int64_t v = 0; v < V; ++v) {
        need(block[v] >= 0, "not stored", V, start, VE, threads, v);
        need(thread[v] == owner_of(v, head, V, VE, threads), "another thread's", V, start, VE, threads, v);
    }
    elements += V;
}

int main() {
    for (int bytes : {2, 4})
        for (int VE : {4, 8})
            for (int threads : {64, 256, 512, 1024}) {
                const int64_t round = (int64_t)threads * VE;
                for (int start : {0, 1, 2, 3, 5, 31, 32, 33, 63})
                    for (int64_t base : {int64_t(1), int64_t(40), round, 2 * round, 4 * round, 5 * round})
                        for (int64_t more : {-64, -33, -8, -7, -4, -1, 0, 1, 3, 4, 7, 8, 33, 64, 70}) {
                            const int64_t V = base + more;
                            if (V < 1) continue;
                            walk(V, start, bytes, VE, threads, 1, V);       // a block to a row
                            for (int64_t cut : {2, 3, 6}) {                 // the backward pass and the cut step
                                const int64_t part = ((V + cut - 1) / cut + round - 1) / round * round;
                                walk(V, start, bytes, VE, threads, (int)((V + part - 1) / part), part);
                            }
                        }
            }
    printf("ok %ld\n", elements);
    return 0;
}
