// Attention over the pages that a cheap score selects: bounds of each page's keys, and the selection.
//
// Bounds.  Over the positions of a page that are inside a sequence, lo_c and hi_c are the smallest and the largest key
// element of channel c, held as whole numbers of 8 bits times one power of two 2^k for the page and head,
//     k = min { k >= -126 : max_c max(|lo_c|, |hi_c|) <= 127 * 2^k },   floor(lo_c 2^-k),   ceil(hi_c 2^-k).
// Score.  The queries of a kv head (its group's heads times the new rows) become whole numbers r of 8 bits with one power of
// two for all of them, rounded to nearest; the score of a page is
//     2^k max_rows sum_c max(r_c lo_c, r_c hi_c),
// which no product of a rounded query with a key of the page exceeds.  The sums are whole numbers below 2^24 and a power of
// two costs nothing, so that scores are exact: the selection does not depend on an order of summation, and equal
// scores go to the page that comes first.
//
// Update: bound by memory, the changed pages' keys read once (and by latency where one page a sequence changes).  A warp
// takes a page and head; its lanes hold 16 bytes of a row each, several rows at once, eight loads under way.
// Select: a cluster of one to eight blocks for each sequence and kv head.  With the negative and the positive parts of a
// query behind one another, a score is one product of 2 d whole numbers, lo first, then hi: m16n8k32 products of 8-bit numbers with
// the rows as the first operand and eight pages as the second.  (This GPU's rate for them is low, and is enough:
// 16 rows of 131K pages and heads took 33 us with four lanes to a page and dp4a.)  A lane's 16 bytes of a page are those
// that it would hold of two steps; the queries are permuted to match.  Scores go to the first block's shared memory, which
// then finds the largest (select.h).
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "device_once.h"
#include "paged_device.h"
#include "select.h"

namespace attn {

namespace {

namespace cg = cooperative_groups;

constexpr int kUpdateThreads = 256;

__device__ __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b) {
    uint32_t y;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    return y;
}
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
    uint32_t y;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    return y;
}
// The smallest k >= -126 with big <= 127 * 2^k for a finite magnitude: 127 = 1.984375 * 2^6.
__device__ __forceinline__ int power_of(uint32_t big) {
    const int k = (int)(big >> 23) - 127 - 6 + ((big & 0x7FFFFFu) > 0x7E0000u ? 1 : 0);
    return max(k, -126);
}
__device__ __forceinline__ float exp2_of(int k) { return __uint_as_float((uint32_t)(k + 127) << 23); }  // -126 .. 127
__device__ __forceinline__ int sequence_length(const PageTable& t, int page, int b, int* err, bool tell) {
    const int n = t.len[b];
    if (n >= 0 && n <= t.max_pages * page) return n;
    if (tell) atomicOr(err, kCacheErrPosition);
    return 0;
}

// A lane's channels of one row, 16 bytes, and the running bounds over rows.
template <bool E4M3>
struct RowBounds;
template <>
struct RowBounds<false> {
    static constexpr int kChannels = 8;
    uint32_t lo[4], hi[4];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo[i] = 0x7F807F80u;
            hi[i] = 0xFF80FF80u;
        }
    }
    __device__ __forceinline__ void take(const uint4& v, uint32_t) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo[i] = min2_nan(lo[i], w[i]);
            hi[i] = max2_nan(hi[i], w[i]);
        }
    }
    __device__ __forceinline__ void join(int o) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo[i] = min2_nan(lo[i], __shfl_xor_sync(0xFFFFFFFFu, lo[i], o));
            hi[i] = max2_nan(hi[i], __shfl_xor_sync(0xFFFFFFFFu, hi[i], o));
        }
    }
    __device__ __forceinline__ void get(float* l, float* h) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            l[2 * i] = __uint_as_float(lo[i] << 16);
            l[2 * i + 1] = __uint_as_float(lo[i] & 0xFFFF0000u);
            h[2 * i] = __uint_as_float(hi[i] << 16);
            h[2 * i + 1] = __uint_as_float(hi[i] & 0xFFFF0000u);
        }
    }
};
// Codes become bf16 numbers: a code's exponent and mantissa, moved to where a bf16 number has them, stand for 2^-120 of it
// (subnormal codes become subnormal numbers), so that two multiplications by powers of two give the row's elements, as exactly
// as a bf16 number can (beyond 2^128: infinities).  (By way of fp16 and float32 numbers 235 MB took 88 us.)
template <>
struct RowBounds<true> {
    static constexpr int kChannels = 16;
    uint32_t lo[8], hi[8];
    uint32_t nan;
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            lo[i] = 0x7F807F80u;
            hi[i] = 0xFF80FF80u;
        }
        nan = 0;
    }
    __device__ __forceinline__ void take(const uint4& v, uint32_t e) {
        // 2^(e - 127) as a bf16 number, twice; for 255 a NaN
        const uint32_t f = (e == 255 ? 0x7FFFu : e == 0 ? 0x0040u : e << 7) * 0x10001u;
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t a = __byte_perm(w[i], 0, 0x1404), b = __byte_perm(w[i], 0, 0x3424);
            uint32_t x = (a & 0x80008000u) | ((a >> 4) & 0x07F007F0u), y = (b & 0x80008000u) | ((b >> 4) & 0x07F007F0u);
            asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(x) : "r"(0x7B807B80u));  // 2^120
            asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(y) : "r"(0x7B807B80u));
            asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(x) : "r"(f));
            asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(y) : "r"(f));
            nan |= ((w[i] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;  // a NaN code: 127 carries into the top bit
            lo[2 * i] = min2_nan(lo[2 * i], x);
            hi[2 * i] = max2_nan(hi[2 * i], x);
            lo[2 * i + 1] = min2_nan(lo[2 * i + 1], y);
            hi[2 * i + 1] = max2_nan(hi[2 * i + 1], y);
        }
    }
    __device__ __forceinline__ void join(int o) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            lo[i] = min2_nan(lo[i], __shfl_xor_sync(0xFFFFFFFFu, lo[i], o));
            hi[i] = max2_nan(hi[i], __shfl_xor_sync(0xFFFFFFFFu, hi[i], o));
        }
    }
    __device__ __forceinline__ void get(float* l, float* h) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            l[2 * i] = nan ? __int_as_float(0x7FFFFFFF) : __uint_as_float(lo[i] << 16);
            l[2 * i + 1] = __uint_as_float(lo[i] & 0xFFFF0000u);
            h[2 * i] = __uint_as_float(hi[i] << 16);
            h[2 * i + 1] = __uint_as_float(hi[i] & 0xFFFF0000u);
        }
    }
};

// The pages of sequence b that hold some of its last new_len positions: [lo, hi).
__device__ __forceinline__ void changed_pages(const BoundsParams& p, int b, bool tell, int& n, int& lo, int& hi) {
    n = sequence_length(p.t, p.c.page, b, p.c.err, tell);
    const int fresh = p.new_len ? max(0, min(p.new_len[b], n)) : n;
    hi = (unsigned)(n + p.c.page - 1) / (unsigned)p.c.page;
    lo = fresh == 0 ? hi : (unsigned)(n - fresh) / (unsigned)p.c.page;
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kUpdateThreads) update_kernel(const __grid_constant__ BoundsParams p) {
    using R = RowBounds<E4M3>;
    constexpr int kLanes = D / R::kChannels;  // of a row
    constexpr int kRows = 32 / kLanes;        // a warp's rows at once
    constexpr int kAhead = 8;
    __shared__ unsigned first[kPagedMaxBatch + 1];  // changed pages of the sequences before b
    __shared__ unsigned scan[kUpdateThreads / 32];
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    wait_for_kernel_before();
    let_kernel_behind_in();
    unsigned carry = 0;
    if (tid == 0) first[0] = 0;
    for (int b0 = 0; b0 < p.B; b0 += kUpdateThreads) {
        const int b = b0 + tid;
        unsigned x = 0;
        if (b < p.B) {
            int n, lo, hi;
            changed_pages(p, b, blockIdx.x == 0, n, lo, hi);
            x = hi - lo;
        }
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const unsigned y = __shfl_up_sync(0xFFFFFFFFu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) scan[warp] = x;
        __syncthreads();
        unsigned all = carry;
#pragma unroll
        for (int w = 0; w < kUpdateThreads / 32; ++w) {
            if (w < warp) x += scan[w];
            all += scan[w];
        }
        if (b < p.B) first[b + 1] = carry + x;
        carry = all;
        __syncthreads();
    }
    const long long items = (long long)carry * p.c.Hkv;
    for (long long item = (long long)blockIdx.x * (kUpdateThreads / 32) + warp; item < items;
         item += (long long)gridDim.x * (kUpdateThreads / 32)) {
        const unsigned entry = (unsigned)(item / p.c.Hkv);
        const int h = (int)(item - (long long)entry * p.c.Hkv);
        int b = 0, top = p.B - 1;  // the last b with first[b] <= entry
        while (b < top) {
            const int mid = (b + top + 1) / 2;
            if (first[mid] <= entry) b = mid;
            else top = mid - 1;
        }
        int n, lo, hi;
        changed_pages(p, b, false, n, lo, hi);
        const int index = lo + (int)(entry - first[b]);
        const int page = p.t.pages[b * p.t.stride + index];
        if (page < 0 || page >= p.c.n_pages) {
            if (lane == 0) atomicOr(p.c.err, kCacheErrPage);
            continue;
        }
        const long long unit = (long long)page * p.c.Hkv + h;
        const int rows = min(p.c.page, n - index * p.c.page), r0 = lane / kLanes;
        const char* src = p.c.pages + unit * 2 * p.c.page * (D * (E4M3 ? 1 : 2)) + 16 * (lane % kLanes);
        const uint8_t* sc = E4M3 ? p.c.scales + unit * (p.c.page / 16) * 32 : nullptr;
        R run;
        run.clear();
        for (int r = r0; r < rows + r0; r += kAhead * kRows) {  // (the same number of rounds for all lanes)
            uint4 v[kAhead];
            uint32_t e[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int row = min(r + i * kRows, rows - 1);  // the last row again changes nothing
                v[i] = *reinterpret_cast<const uint4*>(src + (long long)row * (D * (E4M3 ? 1 : 2)));
                e[i] = E4M3 ? sc[(row / 16) * 32 + row % 16] : 0;
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) run.take(v[i], e[i]);
        }
#pragma unroll
        for (int o = kLanes; o < 32; o *= 2) run.join(o);
        float l[R::kChannels], u[R::kChannels];
        run.get(l, u);
        uint32_t big = 0;  // as bits: a NaN is above an infinity
#pragma unroll
        for (int i = 0; i < R::kChannels; ++i)
            big = max(big, max(__float_as_uint(l[i]) & 0x7FFFFFFFu, __float_as_uint(u[i]) & 0x7FFFFFFFu));
        big = __reduce_max_sync(0xFFFFFFFFu, big);
        const bool bad = big >= 0x7F800000u;
        const int k = bad ? 0 : power_of(big);
        if (lane < kLanes) {
            const float f = exp2_of(-k);
            uint32_t cl[R::kChannels / 4], cu[R::kChannels / 4];
#pragma unroll
            for (int i = 0; i < R::kChannels / 4; ++i) {
                cl[i] = cu[i] = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int a = bad ? 0 : __float2int_rd(l[4 * i + j] * f), c = bad ? 0 : __float2int_ru(u[4 * i + j] * f);
                    cl[i] |= (uint32_t)(a & 0xFF) << 8 * j;
                    cu[i] |= (uint32_t)(c & 0xFF) << 8 * j;
                }
            }
            uint32_t* out = reinterpret_cast<uint32_t*>(p.codes + unit * 2 * D) + lane * (R::kChannels / 4);
#pragma unroll
            for (int i = 0; i < R::kChannels / 4; ++i) {
                out[i] = cl[i];
                out[D / 4 + i] = cu[i];
            }
            if (lane == 0) p.exps[unit] = (uint8_t)(bad ? 255 : k + 127);
        }
    }
}

// ---------------------------------------------------------------------------------------------- selection
constexpr int kSelectThreads = 512;

constexpr int kSelectWarps = kSelectThreads / 32;
template <int D>
struct SelectMemory {
    static constexpr int kPitch = 2 * D + 16;  // rows begin 16 bytes of banks apart
    alignas(16) int8_t q[ATTN_DECODE_MAX_ROWS][kPitch];  // negative parts, positive parts
    SelectShared<kSelectThreads> sel;
    unsigned big[kSelectWarps];
};
__device__ __forceinline__ void mma_s8(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int D, int RT>  // RT: row tiles of 16, at most (the last may be short)
__global__ void __launch_bounds__(kSelectThreads) select_kernel(const __grid_constant__ SelectParams p) {
    __shared__ SelectMemory<D> sh;
    extern __shared__ uint32_t keys[];  // of the first block of the cluster: a page each
    const cg::cluster_group cluster = cg::this_cluster();
    const int blocks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int unit = blockIdx.x / blocks, b = unit / p.Hkv, h = unit - b * p.Hkv, page = p.c.page;
    const int quad = lane / 4, pair = lane % 4;
    wait_for_kernel_before();
    let_kernel_behind_in();
    // the loads that do not wait for one another first: queries, length, the warp's first pages
    const int* row = p.t.pages + b * p.t.stride;
    const uint4* q = reinterpret_cast<const uint4*>(p.q) + (long long)unit * p.rows * (D / 8);
    constexpr int kPieces = (RT * 2 * D + kSelectThreads - 1) / kSelectThreads;  // 16-byte pieces of the queries, a thread's
    uint4 v[kPieces];
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
        const int i = tid + k * kSelectThreads;
        v[k] = i < p.rows * (D / 8) ? q[i] : make_uint4(0, 0, 0, 0);
    }
    constexpr int kAtOnce = RT == 1 ? 2 : 1;  // tiles of eight pages under way
    const int stride = blocks * kSelectWarps * 8 * kAtOnce, lo = p.sinks;
    int i0 = (rank * kSelectWarps + warp) * 8 * kAtOnce;
    int g[kAtOnce];
    auto pages_at = [&](int at) {  // (entries that no position needs may hold anything, and are not used)
#pragma unroll
        for (int x = 0; x < kAtOnce; ++x) g[x] = row[min(lo + at + 8 * x + quad, p.t.max_pages - 1)];
    };
    pages_at(i0);
    const int len = sequence_length(p.t, page, b, p.c.err, tid == 0 && h == 0 && rank == 0);
    const int n = (unsigned)(len + page - 1) / (unsigned)page;
    int* out = p.out_table + (long long)unit * p.keep;
    if (h == 0 && rank == 0 && tid == 0) p.out_len[b] = n > p.keep ? len - (n - p.keep) * page : len;
    if (n <= p.keep) {  // (the whole cluster)
        if (rank == 0)
            for (int i = tid; i < p.keep; i += kSelectThreads) out[i] = i < n ? row[i] : -1;
        return;
    }
    const int m = n - p.recent - lo, K = p.keep - p.recent - lo;  // m > K >= 0
    if (rank == 0) {
        for (int i = tid; i < lo; i += kSelectThreads) out[i] = row[i];
        for (int i = tid; i < p.recent; i += kSelectThreads) out[lo + K + i] = row[n - p.recent + i];
    }
    if (K == 0) return;
    constexpr int kChunks = D / 32;  // 16-byte pieces of a lane and page
    uint4 c[kAtOnce][kChunks];
    uint32_t e[kAtOnce];
    auto codes_of = [&](int at) {
#pragma unroll
        for (int x = 0; x < kAtOnce; ++x) {
            const bool live = at + 8 * x + quad < m, ok = live && g[x] >= 0 && g[x] < p.c.n_pages;
            const long long place = (long long)(ok ? g[x] : 0) * p.Hkv + h;
            const uint4* src = reinterpret_cast<const uint4*>(p.codes + place * 2 * D) + pair;
            e[x] = p.exps[place];
#pragma unroll
            for (int j = 0; j < kChunks; ++j) c[x][j] = src[4 * j];
            if (live && !ok) g[x] = -1;  // told below
            else g[x] = 0;
        }
    };
    codes_of(i0);
    // ---- the queries as whole numbers of one power of two: negative and positive parts
    uint32_t big = 0;  // as bits of a bf16
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
        const uint32_t t = __vmaxu2(__vmaxu2(v[k].x & 0x7FFF7FFFu, v[k].y & 0x7FFF7FFFu),
                                    __vmaxu2(v[k].z & 0x7FFF7FFFu, v[k].w & 0x7FFF7FFFu));
        big = max(big, max(t & 0xFFFFu, t >> 16));
    }
    big = __reduce_max_sync(0xFFFFFFFFu, big);
    if (lane == 0) sh.big[warp] = big;
    __syncthreads();
    big = __reduce_max_sync(0xFFFFFFFFu, sh.big[lane % kSelectWarps]);
    const bool bad = big >= 0x7F80u;  // queries that are not finite choose the first pages
    const float f = bad ? 0.f : exp2_of(-power_of(big << 16));
    const int tiles = (p.rows + 15) / 16;
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {  // (rows up to the end of the last tile: zeros)
        const int i = tid + k * kSelectThreads, r = i / (D / 8), at = i % (D / 8);
        if (r >= 16 * tiles) continue;
        const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
        uint32_t neg[2] = {0, 0}, pos[2] = {0, 0};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float x = __uint_as_float(j % 2 ? w[j / 2] & 0xFFFF0000u : w[j / 2] << 16);
            const int y = bad ? 0 : __float2int_rn(x * f);
            neg[j / 4] |= (uint32_t)(min(y, 0) & 0xFF) << 8 * (j % 4);
            pos[j / 4] |= (uint32_t)max(y, 0) << 8 * (j % 4);
        }
        *reinterpret_cast<uint2*>(&sh.q[r][8 * at]) = make_uint2(neg[0], neg[1]);
        *reinterpret_cast<uint2*>(&sh.q[r][D + 8 * at]) = make_uint2(pos[0], pos[1]);
    }
    if (blocks > 1) cluster.sync();  // (all blocks of the cluster are there)
    else __syncthreads();
    uint32_t* first_keys = blocks > 1 ? cluster.map_shared_rank(keys, 0) : keys;
    uint4 qa[RT == 1 ? kChunks : 1], qb[RT == 1 ? kChunks : 1];  // rows quad and quad + 8
    if constexpr (RT == 1) {
#pragma unroll
        for (int j = 0; j < kChunks; ++j) {
            qa[j] = *reinterpret_cast<const uint4*>(&sh.q[quad][16 * (4 * j + pair)]);
            qb[j] = *reinterpret_cast<const uint4*>(&sh.q[quad + 8][16 * (4 * j + pair)]);
        }
    }
    for (; i0 < m; i0 += stride) {
#pragma unroll
        for (int x = 0; x < kAtOnce; ++x)
            if (g[x] < 0 && h == 0 && pair == 0) atomicOr(p.c.err, kCacheErrPage);
        if (i0 + stride < m) pages_at(i0 + stride);
#pragma unroll
        for (int x = 0; x < kAtOnce; ++x) {
            int best[2] = {-(1 << 30), -(1 << 30)};  // of the lane's rows, for pages 2 pair and 2 pair + 1
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                if (r >= tiles) break;
                int s[4] = {0, 0, 0, 0};
#pragma unroll
                for (int j = 0; j < kChunks; ++j) {
                    uint4 a, b;
                    if constexpr (RT == 1) {
                        a = qa[j];
                        b = qb[j];
                    } else {
                        a = *reinterpret_cast<const uint4*>(&sh.q[16 * r + quad][16 * (4 * j + pair)]);
                        b = *reinterpret_cast<const uint4*>(&sh.q[16 * r + quad + 8][16 * (4 * j + pair)]);
                    }
                    mma_s8(s, a.x, b.x, a.y, b.y, c[x][j].x, c[x][j].y);
                    mma_s8(s, a.z, b.z, a.w, b.w, c[x][j].z, c[x][j].w);
                }
                if (16 * r + quad < p.rows) {
                    best[0] = max(best[0], s[0]);
                    best[1] = max(best[1], s[1]);
                }
                if (16 * r + quad + 8 < p.rows) {
                    best[0] = max(best[0], s[2]);
                    best[1] = max(best[1], s[3]);
                }
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
#pragma unroll
                for (int o = 4; o < 32; o *= 2) best[k] = max(best[k], __shfl_xor_sync(0xFFFFFFFFu, best[k], o));
                const uint32_t ek = __shfl_sync(0xFFFFFFFFu, e[x], 4 * (2 * pair + k));
                const int i = i0 + 8 * x + 2 * pair + k;
                if (quad == k && i < m)
                    first_keys[i] = ek == 255 ? 0xFF800000u : ordered((float)best[k] * __uint_as_float(ek << 23));
            }
        }
        if (i0 + stride < m) codes_of(i0 + stride);
    }
    if (blocks > 1) cluster.sync();
    else __syncthreads();
    if (rank) return;
    select_largest<kSelectThreads, 4>(m, K, sh.sel, [&](int i) { return keys[i]; },
                                   [&](int place, int i) { out[lo + place] = row[lo + i]; });
}

template <class K, class P>
cudaError_t launch_cluster(K* kernel, int grid, int cluster, int threads, int smem, cudaStream_t stream, const P& p) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_bounds_update(const BoundsParams& p, bool e4m3, int n_sm, cudaStream_t stream) {
    const long long items = (long long)p.B * p.t.max_pages * p.c.Hkv, warps = kUpdateThreads / 32;
    const int grid = (int)std::min<long long>((items + warps - 1) / warps, 4LL * n_sm);
    auto go = [&](auto* f) { return launch_dependent(f, dim3((unsigned)grid), kUpdateThreads, 0, stream, p); };
    if (p.c.d == 64) return e4m3 ? go(update_kernel<64, true>) : go(update_kernel<64, false>);
    return e4m3 ? go(update_kernel<128, true>) : go(update_kernel<128, false>);
}

cudaError_t launch_bounds_select(const SelectParams& p, int n_sm, cudaStream_t stream) {
    const int units = p.B * p.Hkv;
    int cluster = 1;  // more blocks while they would be idle and a block has several rounds of pages
    while (cluster < 8 && 2LL * cluster * units <= 2LL * n_sm && p.t.max_pages > cluster * 16 * kSelectWarps) cluster *= 2;
    const int smem = 4 * p.t.max_pages;
    auto go = [&](auto* f) {
        const cudaError_t e = smem_opt_in(reinterpret_cast<const void*>(f), 4 * kSelectMostPages);
        return e != cudaSuccess ? e : launch_cluster(f, units * cluster, cluster, kSelectThreads, smem, stream, p);
    };
    if (p.c.d == 64) return p.rows <= 16 ? go(select_kernel<64, 1>) : go(select_kernel<64, 4>);
    return p.rows <= 16 ? go(select_kernel<128, 1>) : go(select_kernel<128, 4>);
}

}  // namespace attn
