// Rows of a batch that name the same page of a pool.
#pragma once

#include <hip/hip_runtime.h>

namespace dr {

// Whether a row before b, or one after it, names page `slot` too.  Every wave
// scans the list by itself, four slots a lane at a time (one load for 256 rows),
// so that the answer is wave-uniform without a barrier.
__device__ __forceinline__ void slot_sharers(const int* __restrict__ slots, int B, int b, int slot,
                                             bool* earlier, bool* later) {
    const int lane = threadIdx.x & 63;
    bool e = false, l = false;
    for (int i0 = 0; i0 < B; i0 += 256) {
        const int i = i0 + 4 * lane;
        int s[4] = {-1, -1, -1, -1};
        if (i + 3 < B) {
            const int4 v = *reinterpret_cast<const int4*>(slots + i);
            s[0] = v.x; s[1] = v.y; s[2] = v.z; s[3] = v.w;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i + j < B) s[j] = slots[i + j];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            e |= s[j] == slot && i + j < b;
            l |= s[j] == slot && i + j > b;
        }
    }
    *earlier = __ballot(e) != 0;
    *later = __ballot(l) != 0;
}

// The first row after b that names page `slot`, or B.
__device__ __forceinline__ int next_sharer(const int* __restrict__ slots, int B, int b, int slot) {
    for (++b; b < B; ++b)
        if (slots[b] == slot) break;
    return b;
}

}  // namespace dr
