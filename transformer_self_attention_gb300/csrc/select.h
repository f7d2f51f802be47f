// The K largest of n 32-bit keys by one thread block, in the order of their places; of equal keys the first.
//
// The K-th largest key is found digit by digit (11, 11 and 10 bits) from counts in shared memory; then the keys above it,
// and the first of those equal to it, are given out in two sweeps: each warp owns a stretch of neighbouring keys, counts
// what it keeps, and begins where the warps before it end.  Nothing depends on the order in which threads arrive.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace attn {

constexpr int kSelectBins = 2048;

template <int THREADS>
struct SelectShared {
    unsigned count[kSelectBins];
    unsigned scan[THREADS / 32];
    unsigned above[THREADS / 32], equal[THREADS / 32];
    unsigned digit, higher;
};

// Floats as whole numbers in the same order (both zeros are equal; NaN is above everything, whatever its sign).
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFFu;
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// key(i), 0 <= i < n, gives the same number on every call; emit(place, i) is called once for each of the min(n, K) chosen,
// place = 0, 1, .. in the order of i.  All THREADS threads take part.
template <int THREADS, class Key, class Emit>
__device__ __forceinline__ void select_largest(int n, int K, SelectShared<THREADS>& sh, Key key, Emit emit) {
    constexpr int kWarps = THREADS / 32, kPer = kSelectBins / THREADS;
    static_assert(kSelectBins % THREADS == 0, "bins of a thread");
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    if (n <= K) {
        for (int i = tid; i < n; i += THREADS) emit(i, i);
        return;
    }
    if (K <= 0) return;
    uint32_t prefix = 0;
    unsigned want = K;  // of the keys whose upper digits are the prefix
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass < 2 ? 11 : 10;
        for (int i = tid; i < kSelectBins; i += THREADS) sh.count[i] = 0;
        __syncthreads();
        for (int i0 = warp * 32; i0 < n; i0 += THREADS) {
            const int i = i0 + lane;
            bool in = false;
            uint32_t digit = 0;
            if (i < n) {
                const uint32_t k = key(i);
                in = pass == 0 || (k >> (shift + bits)) == prefix;
                digit = k >> shift & ((1u << bits) - 1);
            }
            // all in one bin: a single addition (equal keys would queue up one behind another)
            const unsigned who = __ballot_sync(0xFFFFFFFFu, in);
            if (who == 0) continue;
            const int first = __ffs(who) - 1;
            const uint32_t one = __shfl_sync(0xFFFFFFFFu, digit, first);
            if (__all_sync(0xFFFFFFFFu, !in || digit == one)) {
                if (lane == first) atomicAdd(&sh.count[one], (unsigned)__popc(who));
            } else if (in) {
                atomicAdd(&sh.count[digit], 1u);
            }
        }
        __syncthreads();
        // thread t holds the bins kSelectBins - 1 - kPer t and the kPer - 1 below it
        unsigned mine = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) mine += sh.count[kSelectBins - 1 - kPer * tid - j];
        unsigned upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const unsigned y = __shfl_up_sync(0xFFFFFFFFu, upto, o);
            if (lane >= o) upto += y;
        }
        if (lane == 31) sh.scan[warp] = upto;
        __syncthreads();
        unsigned before = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            if (w < warp) before += sh.scan[w];
        before += upto - mine;  // keys in higher bins than the thread's
        if (before < want && before + mine >= want) {
            int j = 0;
            for (; j < kPer - 1; ++j) {
                const unsigned c = sh.count[kSelectBins - 1 - kPer * tid - j];
                if (before + c >= want) break;
                before += c;
            }
            sh.digit = kSelectBins - 1 - kPer * tid - j;
            sh.higher = before;
        }
        __syncthreads();
        prefix = prefix << bits | sh.digit;
        want -= sh.higher;
    }
    // prefix is the K-th largest key, `want` the number of its equals that are chosen
    const int per = ((n + kWarps - 1) / kWarps + 31) & ~31, from = warp * per, to = min(n, from + per);
    unsigned above = 0, equal = 0;
    for (int i0 = from; i0 < to; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t k = i < to ? key(i) : 0;
        above += __popc(__ballot_sync(0xFFFFFFFFu, i < to && k > prefix));
        equal += __popc(__ballot_sync(0xFFFFFFFFu, i < to && k == prefix));
    }
    if (lane == 0) {
        sh.above[warp] = above;
        sh.equal[warp] = equal;
    }
    __syncthreads();
    above = equal = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
        if (w < warp) {
            above += sh.above[w];
            equal += sh.equal[w];
        }
    unsigned place = above + min(equal, want);
    const unsigned lower = (1u << lane) - 1;
    for (int i0 = from; i0 < to; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t k = i < to ? key(i) : 0;
        const unsigned ties = __ballot_sync(0xFFFFFFFFu, i < to && k == prefix);
        const bool in = i < to && (k > prefix || (k == prefix && equal + __popc(ties & lower) < want));
        const unsigned chosen = __ballot_sync(0xFFFFFFFFu, in);
        if (in) emit((int)(place + __popc(chosen & lower)), i);
        place += __popc(chosen);
        equal += __popc(ties);
    }
}

}  // namespace attn
