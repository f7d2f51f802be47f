// The K largest of n 32-bit keys by one thread block, in the order of their places; of equal keys the first.
//
// First the K-th largest key.  Among up to 256 candidates every thread counts for one of them how many are larger: the K-th
// largest is the smallest that fewer than K exceed.  More keys are brought down to that many by counting them by digits of 11
// bits, from the first bit in which they differ on, and going on with those of the digit that holds the K-th largest: once
// for scores that are alike, twice for weights that spread over many powers of two.  Then the keys above it, and the
// first of those equal to it, are given out: each warp owns a stretch of neighbouring keys, counts what it keeps, and begins
// where the warps before it end.  Nothing depends on the order in which threads arrive.
//
// What it takes are chains of instructions and barriers more than memory: with digits of eight bits all the way, and every warp
// reading the digit off the counts for itself, 91 keys took 4500 cycles and 15K keys 32000.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace attn {

constexpr int kSelectBins = 2048, kSelectFew = 256;

template <int THREADS>
struct SelectShared {
    alignas(16) unsigned count[kSelectBins];
    alignas(16) uint32_t few[kSelectFew];
    unsigned low[THREADS / 32], high[THREADS / 32];
    unsigned digit, higher, inside, n_few, ties;
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
    static_assert(kSelectBins % THREADS == 0 && THREADS >= kSelectFew, "bins of a thread; a candidate each");
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    if (n <= K) {
        for (int i = tid; i < n; i += THREADS) emit(i, i);
        return;
    }
    if (K <= 0) return;
    uint32_t T = 0;     // the K-th largest key,
    unsigned want = K;  // and how many of its equals are chosen
    int few = n;        // candidates
    if (n <= kSelectFew) {
        if (tid < n) sh.few[tid] = key(tid);
    } else {
        uint32_t lo = 0xFFFFFFFFu, hi = 0;
#pragma unroll 4
        for (int i = tid; i < n; i += THREADS) {
            const uint32_t k = key(i);
            lo = min(lo, k);
            hi = max(hi, k);
        }
        lo = __reduce_min_sync(0xFFFFFFFFu, lo);
        hi = __reduce_max_sync(0xFFFFFFFFu, hi);
        if (lane == 0) {
            sh.low[warp] = lo;
            sh.high[warp] = hi;
        }
        __syncthreads();
        lo = __reduce_min_sync(0xFFFFFFFFu, sh.low[lane % kWarps]);
        hi = __reduce_max_sync(0xFFFFFFFFu, sh.high[lane % kWarps]);
        int left = 32 - __clz((int)(hi ^ lo));  // bits that are not known yet
        T = left == 32 ? 0u : hi >> left;       // the bits above them
#pragma unroll 1
        while (left > 0 && few > kSelectFew) {
            const int bits = min(11, left), shift = left - bits;
            const uint32_t mask = (1u << bits) - 1;
#pragma unroll
            for (int j = 0; j < kPer; ++j) sh.count[tid + j * THREADS] = 0;
            __syncthreads();
#pragma unroll 4
            for (int i = tid; i < n; i += THREADS) {
                const uint32_t k = key(i);
                if (left == 32 || k >> left == T) atomicAdd(&sh.count[k >> shift & mask], 1u);
            }
            __syncthreads();
            // thread t has the bins kSelectBins - 1 - kPer t and the kPer - 1 below it
            unsigned c[kPer], mine = 0;
#pragma unroll
            for (int j = 0; j < kPer; ++j) mine += c[j] = sh.count[kSelectBins - 1 - kPer * tid - j];
            unsigned upto = mine;
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const unsigned y = __shfl_up_sync(0xFFFFFFFFu, upto, o);
                if (lane >= o) upto += y;
            }
            if (lane == 31) sh.low[warp] = upto;
            __syncthreads();
            unsigned before = upto - mine + __reduce_add_sync(0xFFFFFFFFu, lane < warp ? sh.low[lane] : 0u);
            if (before < want && before + mine >= want) {
#pragma unroll
                for (int j = 0; j < kPer; ++j) {
                    if (before < want && before + c[j] >= want) {
                        sh.digit = kSelectBins - 1 - kPer * tid - j;
                        sh.higher = before;
                        sh.inside = c[j];
                    }
                    before += c[j];
                }
            }
            if (tid == 0) sh.n_few = 0;
            __syncthreads();
            want -= sh.higher;
            T = T << bits | sh.digit;
            few = sh.inside;
            left = shift;
        }
        if (left > 0) {
            for (int i = tid; i < n; i += THREADS) {
                const uint32_t k = key(i);
                if (k >> left == T) sh.few[atomicAdd(&sh.n_few, 1u)] = k;
            }
        } else {
            few = 0;  // T is known to the last bit
        }
    }
    if (few > 0) {
        __syncthreads();
        const uint32_t k = tid < few ? sh.few[tid] : 0u;
        unsigned more = 0;
        if (warp * 32 < few) {
            int x = 0;
#pragma unroll 4
            for (; x + 4 <= few; x += 4) {
                const uint4 v = *reinterpret_cast<const uint4*>(&sh.few[x]);
                more += (v.x > k) + (v.y > k) + (v.z > k) + (v.w > k);
            }
            for (; x < few; ++x) more += sh.few[x] > k;
        }
        const bool among = tid < few && more < want;
        const uint32_t lowest = __reduce_min_sync(0xFFFFFFFFu, among ? k : 0xFFFFFFFFu);
        if (lane == 0) sh.high[warp] = lowest;
        __syncthreads();
        T = __reduce_min_sync(0xFFFFFFFFu, sh.high[lane % kWarps]);
        if (among && k == T) sh.ties = want - more;
        __syncthreads();
        want = sh.ties;
    }
    const int per = ((n + kWarps - 1) / kWarps + 31) & ~31, from = warp * per, to = min(n, from + per);
    unsigned above = 0, equal = 0;
#pragma unroll 4
    for (int i0 = from; i0 < to; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t k = i < to ? key(i) : 0u;
        above += __popc(__ballot_sync(0xFFFFFFFFu, i < to && k > T));
        equal += __popc(__ballot_sync(0xFFFFFFFFu, i < to && k == T));
    }
    if (lane == 0) {
        sh.count[warp] = above;  // (nobody looks at the counts any more: the barriers above)
        sh.count[kWarps + warp] = equal;
    }
    __syncthreads();
    above = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? sh.count[lane] : 0u);
    equal = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? sh.count[kWarps + lane] : 0u);
    unsigned place = above + min(equal, want);
    const unsigned lower = (1u << lane) - 1;
#pragma unroll 2
    for (int i0 = from; i0 < to; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t k = i < to ? key(i) : 0u;
        const unsigned ties = __ballot_sync(0xFFFFFFFFu, i < to && k == T);
        const bool in = i < to && (k > T || (k == T && equal + __popc(ties & lower) < want));
        const unsigned chosen = __ballot_sync(0xFFFFFFFFu, in);
        if (in) emit((int)(place + __popc(chosen & lower)), i);
        place += __popc(chosen);
        equal += __popc(ties);
    }
}

}  // namespace attn
