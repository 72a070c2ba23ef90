// The bounded wait of the kernels, apart from what it polls, so that it can be
// run on the host as well.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define BL_WAIT_FN __device__ __forceinline__
#else
#define BL_WAIT_FN inline
#endif

namespace bl {

// Poll until poll() is true, giving up once `limit` has passed by now(). A
// thread can be stopped at any place, between a poll that failed and the look
// at the clock too, for longer than the limit; what it waits for may be there
// when it goes on. So the last thing before giving up is a poll, not the clock.
// (One poll: a whole round of them, with a flag for it in the loop, made the
// attention over prompts 2% slower.)
template <int POLLS, class Poll, class Now>
BL_WAIT_FN bool bounded_wait(Poll poll, Now now, uint64_t limit) {
    if (poll()) return true;
    const uint64_t t0 = now();
    for (;;) {
#ifdef __CUDACC__
#pragma unroll 1
#endif
        for (int i = 0; i < POLLS; ++i)
            if (poll()) return true;
        if (now() - t0 > limit) return poll();
    }
}

}  // namespace bl
