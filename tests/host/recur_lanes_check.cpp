// Host check of how the recurrence's channels are dealt to blocks and lanes
// (LaneChannels in kan_token.h): every channel lies in some lane, and leaving
// out what a lane has of the channel block before its own, in the lanes of one
// channel block only.  Exit status 0 and "ok <channels>": everything held.
#include <stdio.h>

#include <vector>

#include "kan_token.h"

using namespace kan;

int main() {
    long channels = 0;
    for (int vec : {1, 4})
        for (int lanes : {4, 8, 16, 32})
            for (int64_t D = vec; D <= 600; ++D) {
                const int64_t blocks = (D + lanes * vec - 1) / (lanes * vec);
                std::vector<int64_t> block(D, -1);
                for (int64_t cb = 0; cb < blocks; ++cb)
                    for (int cl = 0; cl < lanes; ++cl) {
                        const LaneChannels at(cb, cl, lanes, vec, D);
                        for (int i = at.before; i < vec; ++i) {
                            const int64_t c = at.c + i;
                            if (at.c < 0 || c >= D || (block[c] >= 0 && block[c] != cb)) {
                                fprintf(stderr, "vec %d, lanes %d, D %lld: channel %lld in blocks %lld and %lld\n", vec,
                                        lanes, (long long)D, (long long)c, (long long)block[c], (long long)cb);
                                return 1;
                            }
                            block[c] = cb;
                        }
                    }
                for (int64_t c = 0; c < D; ++c)
                    if (block[c] != c / (lanes * vec)) {
                        fprintf(stderr, "channel %lld of %lld is not its block's\n", (long long)c, (long long)D);
                        return 1;
                    }
                channels += D;
            }
    printf("ok %ld\n", channels);
    return 0;
}
