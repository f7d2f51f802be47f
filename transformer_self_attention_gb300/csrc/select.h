// The K largest of n 32-bit keys by one thread block, in the order of their places; of equal keys the first.
//
// The K-th largest key is found digit by digit, eight bits at a time from the first bit in which the keys differ: counts in
// shared memory (those of all passes are cleared at once, so that a pass has one barrier), and every warp reads the digit off
// them for itself.  Then the keys above it, and the first of those equal to it, are given out: each warp owns a
// stretch of neighbouring keys, counts what it keeps, and begins where the warps before it end.  Nothing depends on the
// order in which threads arrive.  Up to HELD keys a thread stay in registers.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace attn {

template <int THREADS>
struct SelectShared {
    alignas(16) unsigned count[4][256];
    unsigned low[THREADS / 32], high[THREADS / 32];
    unsigned above[THREADS / 32], equal[THREADS / 32];
};

// Floats as whole numbers in the same order (both zeros are equal; NaN is above everything, whatever its sign).
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFFu;
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// 0 < K < n.  get(j): the thread's j-th key, that of place warp * per + 32 j + lane (0 where that is not below n).
template <int THREADS, int MOST, class Get, class Emit>
__device__ __forceinline__ void select_from(int n, int K, int per, SelectShared<THREADS>& sh, Get get, Emit emit) {
    constexpr int kWarps = THREADS / 32;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, rounds = per / 32, from = warp * per;
    for (int i = tid; i < 4 * 256; i += THREADS) (&sh.count[0][0])[i] = 0;
    uint32_t lo = 0xFFFFFFFFu, hi = 0;
    auto each = [&](auto&& f) {  // (unrolled where the keys are registers)
        if constexpr (MOST > 0) {
#pragma unroll
            for (int j = 0; j < MOST; ++j)
                if (j < rounds) f(j);
        } else {
            for (int j = 0; j < rounds; ++j) f(j);
        }
    };
    each([&](int j) {
        if (from + 32 * j + lane < n) {
            const uint32_t k = get(j);
            lo = min(lo, k);
            hi = max(hi, k);
        }
    });
    lo = __reduce_min_sync(0xFFFFFFFFu, lo);
    hi = __reduce_max_sync(0xFFFFFFFFu, hi);
    if (lane == 0) {
        sh.low[warp] = lo;
        sh.high[warp] = hi;
    }
    __syncthreads();
    lo = __reduce_min_sync(0xFFFFFFFFu, sh.low[lane % kWarps]);
    hi = __reduce_max_sync(0xFFFFFFFFu, sh.high[lane % kWarps]);
    int left = 32 - __clz((int)(hi ^ lo));                  // bits that are not known yet
    uint32_t prefix = left == 32 ? 0u : hi >> left;         // the bits above them
    unsigned want = K;                                      // of the keys with that prefix
    for (int pass = 0; left > 0; ++pass) {
        const int bits = min(8, left), shift = left - bits;
        const uint32_t mask = (1u << bits) - 1;
        unsigned* count = sh.count[pass];
        each([&](int j) {
            const uint32_t k = get(j);
            const bool in = from + 32 * j + lane < n && (left == 32 || k >> left == prefix);
            const uint32_t digit = k >> shift & mask;
            // all in one bin: a single addition (equal keys would queue up one behind another)
            const unsigned who = __ballot_sync(0xFFFFFFFFu, in);
            if (who == 0) return;
            const int first = __ffs(who) - 1;
            const uint32_t one = __shfl_sync(0xFFFFFFFFu, digit, first);
            if (__all_sync(0xFFFFFFFFu, !in || digit == one)) {
                if (lane == first) atomicAdd(&count[one], (unsigned)__popc(who));
            } else if (in) {
                atomicAdd(&count[digit], 1u);
            }
        });
        __syncthreads();
        // lane l has the bins 255 - 8 l .. 248 - 8 l, from the highest on
        const uint4 a = *reinterpret_cast<const uint4*>(&count[252 - 8 * lane]), b = *reinterpret_cast<const uint4*>(&count[248 - 8 * lane]);
        const unsigned c[8] = {a.w, a.z, a.y, a.x, b.w, b.z, b.y, b.x};
        unsigned mine = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) mine += c[j];
        unsigned upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const unsigned y = __shfl_up_sync(0xFFFFFFFFu, upto, o);
            if (lane >= o) upto += y;
        }
        const int who = __ffs(__ballot_sync(0xFFFFFFFFu, upto >= want)) - 1;  // the lane with the K-th largest
        unsigned before = upto - mine, digit = 0;  // keys in higher bins
        bool found = false;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (!found && before + c[j] >= want) {
                digit = 255 - 8 * lane - j;
                found = true;
            }
            if (!found) before += c[j];
        }
        digit = __shfl_sync(0xFFFFFFFFu, digit, who);
        want -= __shfl_sync(0xFFFFFFFFu, before, who);
        prefix = prefix << bits | digit;
        left = shift;
    }
    // prefix is the K-th largest key, `want` how many of its equals are chosen
    unsigned above = 0, equal = 0;
    each([&](int j) {
        const uint32_t k = get(j);
        const bool live = from + 32 * j + lane < n;
        above += __popc(__ballot_sync(0xFFFFFFFFu, live && k > prefix));
        equal += __popc(__ballot_sync(0xFFFFFFFFu, live && k == prefix));
    });
    if (lane == 0) {
        sh.above[warp] = above;
        sh.equal[warp] = equal;
    }
    __syncthreads();
    const bool earlier = lane < warp && lane < kWarps;
    above = __reduce_add_sync(0xFFFFFFFFu, earlier ? sh.above[lane % kWarps] : 0u);
    equal = __reduce_add_sync(0xFFFFFFFFu, earlier ? sh.equal[lane % kWarps] : 0u);
    unsigned place = above + min(equal, want);
    const unsigned lower = (1u << lane) - 1;
    each([&](int j) {
        const int i = from + 32 * j + lane;
        const uint32_t k = get(j);
        const unsigned ties = __ballot_sync(0xFFFFFFFFu, i < n && k == prefix);
        const bool in = i < n && (k > prefix || (k == prefix && equal + __popc(ties & lower) < want));
        const unsigned chosen = __ballot_sync(0xFFFFFFFFu, in);
        if (in) emit((int)(place + __popc(chosen & lower)), i);
        place += __popc(chosen);
        equal += __popc(ties);
    });
}

// key(i), 0 <= i < n, gives the same number on every call; emit(place, i) is called once for each of the min(n, K) chosen,
// place = 0, 1, .. in the order of i.  All THREADS threads take part.
template <int THREADS, int HELD, class Key, class Emit>
__device__ __forceinline__ void select_largest(int n, int K, SelectShared<THREADS>& sh, Key key, Emit emit) {
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    if (n <= K) {
        for (int i = tid; i < n; i += THREADS) emit(i, i);
        return;
    }
    if (K <= 0) return;
    const int per = ((n + THREADS / 32 - 1) / (THREADS / 32) + 31) & ~31, from = warp * per + lane;
    if (per <= 32 * HELD) {
        uint32_t held[HELD];
#pragma unroll
        for (int j = 0; j < HELD; ++j) held[j] = 32 * j < per && from + 32 * j < n ? key(from + 32 * j) : 0u;
        select_from<THREADS, HELD>(n, K, per, sh, [&](int j) { return held[j]; }, emit);
    } else {
        select_from<THREADS, 0>(n, K, per, sh, [&](int j) { return from + 32 * j < n ? key(from + 32 * j) : 0u; }, emit);
    }
}

}  // namespace attn
