// Device parts the two paged decode kernels share: finding a CTA's work from the lengths on the device.
#pragma once

#include "paged.h"
#include "sm103_ptx.h"

namespace attn {

// Where a warp stands in its CTA's interval of the cost line.  A stretch is the CTA's part of one unit.
struct Walk {
    unsigned at, end;  // cost positions
    int b, h, n;       // current unit (sequence, and kv head or half of its rows) and its key blocks
    int g0, g1;        // the stretch's blocks [g0, g1)
    int lo;            // first key block of the sequence
    int len, seen;     // its visible positions: [seen, len)
};

// A launch that may begin while the kernel before it in the stream still runs; the kernel waits for that one
// (griddepcontrol.wait) before it reads or writes global memory.
template <class K, class... A>
cudaError_t launch_dependent(K* kernel, dim3 grid, int threads, int smem, cudaStream_t stream, const A&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}
__device__ __forceinline__ void wait_for_kernel_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// From here on (in all CTAs) the kernel behind may be brought in; it waits for the end of this one.
__device__ __forceinline__ void let_kernel_behind_in() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// A wait with a limit.  Once one has run out, those of the CTA that are not satisfied return false as well; a loading warp
// then starts no further copies, and the outputs are undefined.
struct Watch {
    volatile int* abort;  // of the CTA, in shared memory
    int* err;
    long long ns;
};
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, const Watch& w) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = ptx::globaltimer();
    while (!ptx::mbar_try_wait(bar, parity)) {
        if (*w.abort) return false;
        if ((long long)(ptx::globaltimer() - t0) > w.ns) {
            *w.abort = 1;
            atomicOr(w.err, kCacheErrWait);
            return false;
        }
    }
    return true;
}
// After an abort, when no warp starts a copy or a product any more: 10 ms for those that are still under way, which write
// shared memory that the next CTA may own.
__device__ __forceinline__ void drain() {
    const uint64_t t0 = ptx::globaltimer();
    while (ptx::globaltimer() - t0 < 10000000ULL) __nanosleep(1000);
}

// Key blocks of sequence b (0 for a length that is not followed).
template <int KEYS>
__device__ __forceinline__ int paged_blocks_of(const PagedParams& p, int n, int& lo) {
    if (n < 0 || n > p.t.max_pages * p.c.page) n = 0;
    int hi;
    paged_blocks(n, p.S_q, p.window, KEYS, lo, hi);
    return hi - lo;
}

// Prefix sums of the sequences' cost of one unit each, cost[0 .. B], by all THREADS of the CTA; scan: a word per warp.
// Returns the sum, and in `busy` the number of sequences with keys.
template <int KEYS, int THREADS>
__device__ __forceinline__ unsigned paged_prefix(const PagedParams& p, PagedShape shape, unsigned* cost, unsigned* scan,
                                                 int& busy) {
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    unsigned carry = 0;
    busy = 0;
    if (tid == 0) cost[0] = 0;
    for (int b0 = 0; b0 < p.B; b0 += THREADS) {
        const int b = b0 + tid;
        unsigned x = 0;
        if (b < p.B) {
            const int len = p.t.len[b];
            int lo;
            x = paged_cost(paged_blocks_of<KEYS>(p, len, lo), shape);
            if (blockIdx.x == 0 && (len < 0 || len > p.t.max_pages * p.c.page)) atomicOr(p.c.err, kCacheErrPosition);
        }
        const bool some = x != 0;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const unsigned y = __shfl_up_sync(0xFFFFFFFFu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) scan[warp] = x;
        busy += __syncthreads_count(some);
        unsigned before = carry, all = carry;
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) {
            if (w < warp) before += scan[w];
            all += scan[w];
        }
        if (b < p.B) cost[b + 1] = before + x;
        carry = all;
        __syncthreads();
    }
    return carry;
}

// The CTA's share of the sequences without keys: rows of zeros, LSE -inf, nothing to join.
template <int D, int THREADS>
__device__ __forceinline__ void paged_empty_rows(const PagedParams& p, const unsigned* cost) {
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        if (cost[b + 1] != cost[b]) continue;
        if (p.by_unit)
            for (int i = threadIdx.x; i < p.units; i += THREADS) p.cut[b * p.units + i] = make_int2(-1, 0);
        if (p.whole_o) {
            for (int i = threadIdx.x; i < p.Hq * p.S_q; i += THREADS)
                p.whole_ml[(long long)b * p.Hq * p.S_q + i] = make_float2(__int_as_float(0xFF800000), 0.f);
            continue;
        }
        uint4* o = reinterpret_cast<uint4*>(p.o) + (long long)b * p.Hq * p.S_q * (D / 8);
        for (int i = threadIdx.x; i < p.Hq * p.S_q * (D / 8); i += THREADS) o[i] = make_uint4(0, 0, 0, 0);
        if (p.lse)
            for (int i = threadIdx.x; i < p.Hq * p.S_q; i += THREADS)
                p.lse[(long long)b * p.Hq * p.S_q + i] = __int_as_float(0xFF800000);
    }
}

__device__ __forceinline__ Walk paged_begin(const PagedParams& p, const PagedCuts& cuts, const unsigned* cost) {
    Walk w{};
    w.at = cuts.begin(blockIdx.x);
    w.end = cuts.begin(blockIdx.x + 1);
    int lo = 0, hi = p.B - 1;  // the last b whose cost begins at or before w.at
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (cost[mid] * p.units <= w.at) lo = mid;
        else hi = mid - 1;
    }
    w.b = lo;
    return w;
}

// The stretch that begins at w.at: its unit, its blocks (none, where the interval covers a unit's overhead alone), and
// w.at moved behind it.
template <int KEYS>
__device__ __forceinline__ void paged_open(const PagedParams& p, PagedShape shape, const unsigned* cost, Walk& w) {
    while (cost[w.b + 1] * p.units <= w.at) ++w.b;
    w.len = p.t.len[w.b];
    w.n = paged_blocks_of<KEYS>(p, w.len, w.lo);
    w.seen = p.window < 0 ? 0 : max(0, w.len - p.S_q - p.window);
    const unsigned into = w.at - cost[w.b] * p.units, per = paged_cost(w.n, shape);
    w.h = (int)(into / per);
    const unsigned off = into - w.h * per, to = min(per, off + (w.end - w.at));
    w.g0 = min(w.n, max(0, (int)off - (int)shape.overhead));
    w.g1 = min(w.n, max(0, (int)to - (int)shape.overhead));
    w.at += to - off;
}

// Records a unit for the joining kernel (one thread, of the CTA w in which the unit begins; final: it also ends there).
__device__ __forceinline__ void paged_record_cut(const PagedParams& p, const PagedCuts& cuts, PagedShape shape,
                                                 const unsigned* cost, const Walk& w, bool final) {
    const int unit = w.b * p.units + w.h;
    if (final) {
        if (p.by_unit) p.cut[unit] = make_int2(-1, 0);
        return;
    }
    const unsigned u0 = cost[w.b] * p.units + w.h * paged_cost(w.n, shape) + shape.overhead;
    const int last = (int)cuts.owner(u0 + w.n - 1);
    if (p.by_unit) p.cut[unit] = make_int2((int)blockIdx.x, last);
    else p.cut[blockIdx.x] = make_int2(unit, last);
}

// Four floats of magnitude at most 448 as two E4M3 numbers each, x = hi + lo / 16: hi has four significant bits, the
// remainder is taken exactly, and lo has four bits of it (down to steps of 2^-9 / 16).
__device__ __forceinline__ void split_e4m3(float x0, float x1, float x2, float x3, uint32_t& hi, uint32_t& lo) {
    hi = ptx::pack_e4m3x4(x0, x1, x2, x3);
    uint32_t h01, h23;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h01) : "h"((uint16_t)hi));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h23) : "h"((uint16_t)(hi >> 16)));
    float f0, f1, f2, f3;
    asm("{.reg .f16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b;}" : "=f"(f0), "=f"(f1) : "r"(h01));
    asm("{.reg .f16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b;}" : "=f"(f2), "=f"(f3) : "r"(h23));
    lo = ptx::pack_e4m3x4((x0 - f0) * 16.f, (x1 - f1) * 16.f, (x2 - f2) * 16.f, (x3 - f3) * 16.f);
}

}  // namespace attn
