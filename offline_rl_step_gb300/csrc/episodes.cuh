// Packed episodes seen from a range of tokens: which tokens begin an episode.
//
// Kernels that cut the packed tokens into ranges of their own size, whatever
// the episodes are, need for each range the episode its first token is in and
// the tokens at which an episode begins.  Every access stays in bounds whatever
// the ends hold, and every loop ends.
#pragma once

#include <stdint.h>

namespace ofrl {

__device__ __forceinline__ int episode_end(const int32_t* ends, int e, int tokens) {
    return min(max(ends[e], 0), tokens);
}
__device__ __forceinline__ int episode_start(const int32_t* ends, int e, int tokens) {
    return e > 0 ? episode_end(ends, e - 1, tokens) : 0;
}

// The first episode from `lo` on that ends after token t (the one t is in), or
// `episodes`: a search that cuts the range into 32 each round.  One whole warp.
__device__ __forceinline__ int find_episode(const int32_t* ends, int lo, int episodes, int tokens, int t) {
    const int lane = threadIdx.x & 31;
    int hi = episodes;
    while (hi > lo) {
        const int step = (int)(((int64_t)hi - lo + 31) / 32);
        const int at = (int)min((int64_t)lo + (int64_t)(lane + 1) * step, (int64_t)hi) - 1;
        const unsigned m = __ballot_sync(0xffffffffu, episode_end(ends, at, tokens) > t);
        if (m == 0) return hi;
        const int f = __ffs(m) - 1;
        hi = __shfl_sync(0xffffffffu, at, f);
        lo = (int)min((int64_t)lo + (int64_t)f * step, (int64_t)hi);
    }
    return lo;
}

// The next episode after e that ends after token t, or `episodes`: looks at 32
// at a time, since it is nearly always the next one.  One whole warp.
__device__ __forceinline__ int next_episode(const int32_t* ends, int e, int episodes, int tokens, int t) {
    const int lane = threadIdx.x & 31;
    for (int base = e + 1; base < episodes; base += 32) {
        const unsigned m = __ballot_sync(0xffffffffu, lane < episodes - base &&
                                                          episode_end(ends, min(base + lane, episodes - 1), tokens) > t);
        if (m) return base + __ffs(m) - 1;
        if (episodes - base <= 32) break;
    }
    return episodes;
}

// Tokens [s0, s1) of a call.
struct Range {
    int e0;            // the episode token s0 is in, or `episodes`
    int end;           // tokens from here on (below s1) belong to no episode
    int closed;        // 1: an episode ends with token end - 1
};

// One whole warp: the range's facts, and bit i of mask (shared memory, zeroed,
// (s1 - s0 + 31) / 32 words) set where token s0 + i begins an episode.
__device__ __forceinline__ Range mark_starts(const int32_t* ends, int episodes, int tokens, int s0, int s1,
                                             uint32_t* mask) {
    const int lane = threadIdx.x & 31;
    const int live = episodes > 0 ? episode_end(ends, episodes - 1, tokens) : 0;
    Range r;
    r.e0 = find_episode(ends, 0, episodes, tokens, s0);
    r.end = max(min(s1, live), s0);
    bool closed = r.end == live;
    if (lane == 0 && r.e0 < episodes && episode_start(ends, r.e0, tokens) == s0) atomicOr(mask, 1u);
    for (int base = r.e0; base < episodes; base += 32) {
        const int v = lane < episodes - base ? episode_end(ends, base + lane, tokens) : INT32_MAX;
        if (v > s0 && v < r.end) atomicOr(mask + ((v - s0) >> 5), 1u << ((v - s0) & 31));
        closed = closed || __any_sync(0xffffffffu, v == r.end);
        if (__any_sync(0xffffffffu, v > r.end) || episodes - base <= 32) break;
    }
    r.closed = closed;
    return r;
}

// Ends that lie below their predecessor or outside [0, tokens], of every
// step-th block of 32 from the first-th on.  One whole warp; lane 0's count.
__device__ __forceinline__ int count_bad_ends(const int32_t* ends, int episodes, int tokens, int first, int step) {
    const int lane = threadIdx.x & 31;
    int bad = 0;
    for (int64_t base = (int64_t)first * 32; base < episodes; base += (int64_t)step * 32) {
        const int64_t e = base + lane;
        if (e < episodes) {
            const int32_t v = ends[e];
            bad += v < (e > 0 ? ends[e - 1] : 0) || v > tokens;
        }
    }
    for (int o = 16; o > 0; o >>= 1) bad += __shfl_down_sync(0xffffffffu, bad, o);
    return bad;
}

}  // namespace ofrl
