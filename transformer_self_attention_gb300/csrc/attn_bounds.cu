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
// Update: bound by memory, the changed pages' keys read once, or by latency where one page a sequence changes.  A warp takes
// a page and head, or the whole block does where there are fewer of them than blocks; the lanes hold 16 bytes of a row
// each, several rows at once, eight loads under way, and the next page's are begun before this one's bounds are
// joined and written (235 MB of codes: 56 us with all lanes joining all channels and nothing ahead, 44 so; 470 MB of bf16
// keys 74 us).  Pages of 16 positions are bound by instructions: 158 us for 235 MB of codes with d 64, 95 with d 128.
// Select: a cluster of one to eight blocks for each sequence and kv head.  With the negative and the positive parts of a
// query behind one another, a score is one product of 2 d whole numbers, lo first, then hi: m16n8k16 products of fp16 numbers,
// which hold them exactly, as float32 holds their sums, with the rows as the first operand and eight pages as the second.
// (Products of 8-bit whole numbers, m16n8k32, took 200 cycles each, and dp4a with four lanes to a page was no faster.)  A
// lane's 16 bytes of a page are those that it would hold of four steps; the queries are permuted to match.  Scores go to the
// first block's shared memory, which then finds the largest (select.h).
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "device_once.h"
#include "paged_device.h"
#include "select.h"

namespace attn {

namespace {

namespace cg = cooperative_groups;

constexpr int kUpdateThreads = 256;
__host__ __device__ constexpr int update_blocks(bool e4m3) { return e4m3 ? 3 : 4; }  // of a multiprocessor, all at once

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

// A lane's channels of one row, 16 bytes, and the running bounds over rows: bf16.
struct RowBounds {
    static constexpr int kChannels = 8;
    uint32_t lo[4], hi[4];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo[i] = 0x7F807F80u;
            hi[i] = 0xFF80FF80u;
        }
    }
    __device__ __forceinline__ void take(const uint4& v, uint32_t, uint32_t) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo[i] = least(lo[i], w[i]);
            hi[i] = most(hi[i], w[i]);
        }
    }
    static __device__ __forceinline__ uint32_t least(uint32_t a, uint32_t b) { return min2_nan(a, b); }
    static __device__ __forceinline__ uint32_t most(uint32_t a, uint32_t b) { return max2_nan(a, b); }
    static __device__ __forceinline__ float2 value(uint32_t w, uint32_t) {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    }
};
// E4M3: both bounds of a pair of channels as packed 16-bit numbers.  Where the rows' exponents lie within 14 of the largest
// (WIDE false), codes become fp16 numbers times 2^(e - largest), exactly; otherwise bf16 numbers: a code's exponent and
// mantissa, moved to where a bf16 number has them, stand for 2^-120 of it (subnormal codes become subnormal numbers), and two
// multiplications by powers of two give the element, as exactly as a bf16 number can (beyond 2^128: infinities).  The second
// form takes twice the instructions: 69 against 44 us for 235 MB (d 128, pages of 64).
template <bool WIDE>
struct CodeBounds {
    static constexpr int kChannels = 16;
    uint32_t lo[8], hi[8];
    uint32_t nan;
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            lo[i] = WIDE ? 0x7F807F80u : 0x7C007C00u;
            hi[i] = WIDE ? 0xFF80FF80u : 0xFC00FC00u;
        }
        nan = 0;
    }
    static __device__ __forceinline__ uint32_t least(uint32_t a, uint32_t b) {
        uint32_t y;
        if constexpr (WIDE) asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
        else asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
        return y;
    }
    static __device__ __forceinline__ uint32_t most(uint32_t a, uint32_t b) {
        uint32_t y;
        if constexpr (WIDE) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
        else asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
        return y;
    }
    __device__ __forceinline__ void take(const uint4& v, uint32_t e, uint32_t top) {
        // 2^(e - 127) as a bf16 number, or 2^(e - top) as an fp16 number, twice (no row has 255 here)
        const uint32_t f = (WIDE ? (e == 0 ? 0x0040u : e << 7) : e + 15 - top << 10) * 0x10001u;
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t x, y;
            if constexpr (WIDE) {
                const uint32_t a = __byte_perm(w[i], 0, 0x1404), b = __byte_perm(w[i], 0, 0x3424);
                x = (a & 0x80008000u) | ((a >> 4) & 0x07F007F0u);
                y = (b & 0x80008000u) | ((b >> 4) & 0x07F007F0u);
                asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(x) : "r"(0x7B807B80u));  // 2^120
                asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(y) : "r"(0x7B807B80u));
                asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(x) : "r"(f));
                asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(y) : "r"(f));
                nan |= ((w[i] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;  // a NaN code: 127 carries into the top bit
            } else {
                asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(x) : "h"((uint16_t)w[i]));
                asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(y) : "h"((uint16_t)(w[i] >> 16)));
                asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(x) : "r"(f));
                asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(y) : "r"(f));
            }
            lo[2 * i] = least(lo[2 * i], x);
            hi[2 * i] = most(hi[2 * i], x);
            lo[2 * i + 1] = least(lo[2 * i + 1], y);
            hi[2 * i + 1] = most(hi[2 * i + 1], y);
        }
    }
    static __device__ __forceinline__ float2 value(uint32_t w, uint32_t top) {
        if constexpr (WIDE) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
        const float f = __uint_as_float(max(top << 23, 0x00400000u));
        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w));
        return make_float2(x.x * f, x.y * f);
    }
};

// The pages of sequence b that hold some of its last new_len positions: [lo, hi).
__device__ __forceinline__ void changed_pages(const BoundsParams& p, int b, bool tell, int& n, int& lo, int& hi) {
    n = sequence_length(p.t, p.c.page, b, p.c.err, tell);
    const int fresh = p.new_len ? max(0, min(p.new_len[b], n)) : n;
    hi = (unsigned)(n + p.c.page - 1) / (unsigned)p.c.page;
    lo = fresh == 0 ? hi : (unsigned)(n - fresh) / (unsigned)p.c.page;
}

// The bounds of one page and head by `share` warps (1, or all of the block, which then meet in `joint`); `part`: the warp's
// number among them.
template <int D, bool E4M3>
struct Rows {  // a warp's loads of some rows: 16 bytes a lane and row
    static constexpr int kRow = D * (E4M3 ? 1 : 2), kLanes = kRow / 16, kAtOnce = 32 / kLanes, kAhead = 8;
    static constexpr int kRound = kAhead * kAtOnce;
    uint4 v[kAhead];
    uint32_t e[kAhead];
    int used;  // of them
    __device__ __forceinline__ void load(const BoundsParams& p, long long unit, int rows, int r0) {
        const int lane = threadIdx.x % 32;
        const char* src = p.c.pages + unit * 2 * p.c.page * kRow + 16 * (lane % kLanes);
        const uint8_t* sc = E4M3 ? p.c.scales + unit * (p.c.page / 16) * 32 : nullptr;
        used = E4M3 ? min(kAhead, (rows - r0 + kAtOnce - 1) / kAtOnce) : kAhead;
        if (r0 % 16 == 0 && r0 + kRound <= rows) {  // one address, and constants
            src += (r0 + lane / kLanes) * (long long)kRow;
            if (E4M3) sc += r0 * 2 + lane / kLanes;
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                v[i] = *reinterpret_cast<const uint4*>(src + i * kAtOnce * kRow);
                e[i] = E4M3 ? sc[i * kAtOnce / 16 * 32 + i * kAtOnce % 16] : 0;
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (E4M3 && i >= used) break;
            const int row = min(r0 + i * kAtOnce + lane / kLanes, rows - 1);  // the last row again changes nothing
            v[i] = *reinterpret_cast<const uint4*>(src + (long long)row * kRow);
            e[i] = E4M3 ? sc[(row / 16) * 32 + row % 16] : 0;
        }
    }
};
// `ahead` starts the loads of the page behind this one.
template <int D, bool E4M3, class R, class F>
__device__ __forceinline__ void page_bounds(const BoundsParams& p, long long unit, int rows, uint32_t top, int part, int share,
                                            Rows<D, E4M3>& x, uint32_t (*joint)[2][32][2], F ahead) {
    using X = Rows<D, E4M3>;
    constexpr int kLanes = X::kLanes, kWords = R::kChannels / 2;
    const int lane = threadIdx.x % 32;
    R run;
    run.clear();
    for (int r0 = part * X::kRound; r0 < rows;) {  // (the first rows have been loaded)
        if (!E4M3 || x.used == X::kAhead) {
#pragma unroll
            for (int i = 0; i < X::kAhead; ++i) run.take(x.v[i], x.e[i], top);
        } else {
#pragma unroll
            for (int i = 0; i < X::kAhead - 1; ++i)
                if (i < x.used) run.take(x.v[i], x.e[i], top);
        }
        r0 += share * X::kRound;
        if (r0 < rows) x.load(p, unit, rows, r0);
    }
    ahead();
    // over the lanes that hold the same channels of other rows, which are left with half of the channels after each step
    uint32_t(&l)[kWords] = run.lo, (&h)[kWords] = run.hi;
    int first = 0;  // of the lane's words
#pragma unroll
    for (int o = kLanes, n = kWords / 2; o < 32; o *= 2, n /= 2) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const uint32_t l_in = __shfl_xor_sync(0xFFFFFFFFu, up ? l[i] : l[n + i], o);
            const uint32_t h_in = __shfl_xor_sync(0xFFFFFFFFu, up ? h[i] : h[n + i], o);
            l[i] = R::least(up ? l[n + i] : l[i], l_in);
            h[i] = R::most(up ? h[n + i] : h[i], h_in);
        }
        first += up ? n : 0;
    }
    constexpr int kMine = kWords * kLanes / 32;  // words of a lane now: D channels over the warp
    static_assert(kMine == 1 || kMine == 2, "channels of a lane");
    bool nan = false;
    if constexpr (E4M3) nan = run.nan != 0;
    if (share > 1) {
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            joint[part][0][lane][i] = l[i];
            joint[part][1][lane][i] = h[i];
        }
        nan = __syncthreads_or(nan);
        if (part) return;
        for (int w = 1; w < share; ++w)
#pragma unroll
            for (int i = 0; i < kMine; ++i) {
                l[i] = R::least(l[i], joint[w][0][lane][i]);
                h[i] = R::most(h[i], joint[w][1][lane][i]);
            }
    }
    uint32_t big = nan ? 0x7FFFFFFFu : 0;  // as bits: a NaN is above an infinity
    float2 u[kMine], v[kMine];
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        u[i] = R::value(l[i], top);
        v[i] = R::value(h[i], top);
        for (const float y : {u[i].x, u[i].y, v[i].x, v[i].y}) big = max(big, __float_as_uint(y) & 0x7FFFFFFFu);
    }
    big = __reduce_max_sync(0xFFFFFFFFu, big);
    const bool bad = big >= 0x7F800000u;
    const int k = bad ? 0 : power_of(big);
    const float f = exp2_of(-k);
    uint32_t below = 0, above = 0;
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const int a = __float2int_rd(u[i].x * f), b = __float2int_rd(u[i].y * f);
        const int c = __float2int_ru(v[i].x * f), d = __float2int_ru(v[i].y * f);
        below |= (uint32_t)((a & 0xFF) | (b & 0xFF) << 8) << 16 * i;
        above |= (uint32_t)((c & 0xFF) | (d & 0xFF) << 8) << 16 * i;
    }
    if (bad) below = above = 0;
    int8_t* out = p.codes + unit * 2 * D + lane % kLanes * R::kChannels + 2 * first;
    if constexpr (kMine == 2) {
        *reinterpret_cast<uint32_t*>(out) = below;
        *reinterpret_cast<uint32_t*>(out + D) = above;
    } else {
        *reinterpret_cast<uint16_t*>(out) = (uint16_t)below;
        *reinterpret_cast<uint16_t*>(out + D) = (uint16_t)above;
    }
    if (lane == 0) p.exps[unit] = (uint8_t)(bad ? 255 : k + 127);
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kUpdateThreads, update_blocks(E4M3)) update_kernel(const __grid_constant__ BoundsParams p) {
    constexpr int kWarps = kUpdateThreads / 32;
    __shared__ uint32_t joint[kWarps][2][32][2];
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
    const unsigned items = carry * p.c.Hkv;
    const unsigned share = items <= gridDim.x ? kWarps : 1, part = share > 1 ? warp : 0, step = gridDim.x * kWarps / share;
    // The warp's items, `step` apart: the page of the next one is looked at an item later.
    struct Item {
        int page, h, rows;
    };
    unsigned item = (blockIdx.x * kWarps + warp) / share;
    auto look_up = [&] {
        Item x{0, 0, 0};
        if (item >= items) return x;
        const unsigned entry = item / (unsigned)p.c.Hkv;
        int b = 0, top = p.B - 1;  // the last b with first[b] <= entry
        while (b < top) {
            const int mid = (b + top + 1) / 2;
            if (first[mid] <= entry) b = mid;
            else top = mid - 1;
        }
        int n, lo, hi;
        changed_pages(p, b, false, n, lo, hi);
        const int index = lo + (int)(entry - first[b]);
        x.page = p.t.pages[b * p.t.stride + index];
        x.h = (int)(item - entry * (unsigned)p.c.Hkv);
        x.rows = min(p.c.page, n - index * p.c.page);
        item += step;
        return x;
    };
    Rows<D, E4M3> x;
    uint32_t e[2];  // E4M3: exponents of rows `lane` and 32 + `lane`
    auto good = [&](const Item& i) { return i.page >= 0 && i.page < p.c.n_pages; };
    auto load = [&](const Item& i) {
        if (i.rows <= 0 || !good(i)) return;
        const long long unit = (long long)i.page * p.c.Hkv + i.h;
        x.load(p, unit, i.rows, min(part * Rows<D, E4M3>::kRound, i.rows - 1));
        if constexpr (E4M3) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int r = min(32 * k + lane, i.rows - 1);
                e[k] = p.c.scales[unit * (p.c.page / 16) * 32 + (r / 16) * 32 + r % 16];
            }
        }
    };
    Item now = look_up(), next;
    load(now);
    for (; now.rows > 0; now = next) {
        next = look_up();
        if (!good(now)) {
            if (lane == 0) atomicOr(p.c.err, kCacheErrPage);
            load(next);
            continue;  // (all warps that share the page)
        }
        const int rows = now.rows;
        const long long unit = (long long)now.page * p.c.Hkv + now.h;
        auto ahead = [&] { load(next); };
        if constexpr (E4M3) {
            // the largest and the smallest exponent of the rows
            const uint8_t* sc = p.c.scales + unit * (p.c.page / 16) * 32;
            uint32_t most = max(e[0], e[1]), least = min(e[0], e[1]);
            for (int r = 64 + lane; r < rows; r += 32) {
                const uint32_t y = sc[(r / 16) * 32 + r % 16];
                most = max(most, y);
                least = min(least, y);
            }
            most = __reduce_max_sync(0xFFFFFFFFu, most);
            least = __reduce_min_sync(0xFFFFFFFFu, least);
            if (most == 255) {  // a row that is not finite
                if (part == 0) {
                    for (int i = lane; i < 2 * D / 4; i += 32) reinterpret_cast<uint32_t*>(p.codes + unit * 2 * D)[i] = 0;
                    if (lane == 0) p.exps[unit] = 255;
                }
                load(next);
            } else if (most - least <= 14) {
                page_bounds<D, true, CodeBounds<false>>(p, unit, rows, most, part, share, x, joint, ahead);
            } else {
                page_bounds<D, true, CodeBounds<true>>(p, unit, rows, most, part, share, x, joint, ahead);
            }
        } else {
            page_bounds<D, false, RowBounds>(p, unit, rows, 0, part, share, x, joint, ahead);
        }
        if (share > 1) __syncthreads();
    }
}

// ---------------------------------------------------------------------------------------------- selection
constexpr int kSelectThreads = 256, kSelectBlocks = 3;  // a multiprocessor: with 512 threads one block fitted, 24 us for 512 heads

constexpr int kSelectWarps = kSelectThreads / 32;
template <int D, int RT>
struct SelectMemory {
    static constexpr int kPitch = 4 * D + 16;  // bytes; rows begin 16 bytes of banks apart
    alignas(16) uint8_t q[RT * 16][kPitch];    // negative parts, positive parts, fp16
    SelectShared<kSelectThreads> sel;
    unsigned big[kSelectWarps];
};
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Four whole numbers of 8 bits as fp16 numbers: with the sign turned they are 0 .. 255 above -128, and 1024 + that has them as
// its last bits.
__device__ __forceinline__ void widen_s8(uint32_t w, uint32_t& lo, uint32_t& hi) {
    const uint32_t u = w ^ 0x80808080u;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(__byte_perm(u, 0x64646464u, 0x4140)), "r"(0x64806480u));  // 1152
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(__byte_perm(u, 0x64646464u, 0x4342)), "r"(0x64806480u));
}
__device__ __forceinline__ uint32_t f16_pair(float lo, float hi) {
    uint32_t y;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
    return y;
}

template <int D, int RT>  // RT: row tiles of 16, at most (the last may be short)
__global__ void __launch_bounds__(kSelectThreads, RT == 1 ? kSelectBlocks : 2) select_kernel(const __grid_constant__ SelectParams p) {
    __shared__ SelectMemory<D, RT> sh;
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
    // a warp's round: a tile of eight pages, one for each four lanes
    const int stride = blocks * kSelectWarps * 8, lo = p.sinks;
    int i0 = (rank * kSelectWarps + warp) * 8;
    auto page_at = [&](int i) { return row[min(lo + i + quad, p.t.max_pages - 1)]; };  // (beyond those in use: anything)
    int g = page_at(i0), g1 = page_at(i0 + stride), g2 = page_at(i0 + 2 * stride);  // this round's, and the next ones'
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
    uint4 c[kChunks];
    uint32_t e = 0;
    bool astray = false;
    auto place_of = [&](int page_no, int i) {
        const bool live = i + quad < m, ok = live && page_no >= 0 && page_no < p.c.n_pages;
        astray |= live && !ok;
        return (long long)(ok ? page_no : 0) * p.Hkv + h;
    };
    auto codes_of = [&](int page_no, int i) {
        const long long place = place_of(page_no, i);
        const uint4* src = reinterpret_cast<const uint4*>(p.codes + place * 2 * D) + pair;
        e = p.exps[place];
#pragma unroll
        for (int j = 0; j < kChunks; ++j) c[j] = src[4 * j];
    };
    auto to_l2 = [&](int page_no, int i) {  // (2 d bytes: a line of 128 to a lane)
        if (i < m && pair < 2 * D / 128)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(p.codes + place_of(page_no, i) * 2 * D + 128 * pair));
    };
    codes_of(g, i0);
    to_l2(g1, i0 + stride);
    to_l2(g2, i0 + 2 * stride);
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
    const bool bad = big >= 0x7F80u;  // not finite: zeros (the first pages, behind those of exponent 255)
    const float f = bad ? 0.f : exp2_of(-power_of(big << 16));
    const int tiles = (p.rows + 15) / 16;
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {  // (rows up to the end of the last tile: zeros)
        const int i = tid + k * kSelectThreads, r = i / (D / 8), at = i % (D / 8);
        if (r >= 16 * tiles) continue;
        const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
        uint32_t neg[4], pos[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float x = bad ? 0.f : rintf(__uint_as_float(w[j] << 16) * f);
            const float y = bad ? 0.f : rintf(__uint_as_float(w[j] & 0xFFFF0000u) * f);
            neg[j] = f16_pair(fminf(x, 0.f), fminf(y, 0.f));
            pos[j] = f16_pair(fmaxf(x, 0.f), fmaxf(y, 0.f));
        }
        *reinterpret_cast<uint4*>(&sh.q[r][16 * at]) = make_uint4(neg[0], neg[1], neg[2], neg[3]);
        *reinterpret_cast<uint4*>(&sh.q[r][2 * D + 16 * at]) = make_uint4(pos[0], pos[1], pos[2], pos[3]);
    }
    if (blocks > 1) cluster.sync();  // (all blocks of the cluster are there)
    else __syncthreads();
    uint32_t* first_keys = blocks > 1 ? cluster.map_shared_rank(keys, 0) : keys;
    for (; i0 < m; i0 += stride) {
        float best[2] = {-16777216.f, -16777216.f};  // of the lane's rows, for pages 2 pair and 2 pair + 1
#pragma unroll 1
        for (int r = 0; r < tiles; ++r) {
            float s[2][4];  // two chains
#pragma unroll
            for (int k = 0; k < 4; ++k) s[0][k] = s[1][k] = 0.f;
#pragma unroll
            for (int j = 0; j < kChunks; ++j) {
                const uint8_t* qa = &sh.q[16 * r + quad][32 * (4 * j + pair)];
                const uint8_t* qb = &sh.q[16 * r + quad + 8][32 * (4 * j + pair)];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const uint4 a = *reinterpret_cast<const uint4*>(qa + 16 * y), b = *reinterpret_cast<const uint4*>(qb + 16 * y);
                    uint32_t b0, b1, b2, b3;
                    widen_s8(y ? c[j].z : c[j].x, b0, b1);
                    widen_s8(y ? c[j].w : c[j].y, b2, b3);
                    mma_f16(s[0], a.x, b.x, a.y, b.y, b0, b1);
                    mma_f16(s[1], a.z, b.z, a.w, b.w, b2, b3);
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (16 * r + quad + 8 * (k / 2) < p.rows) best[k % 2] = fmaxf(best[k % 2], s[0][k] + s[1][k]);
        }
        const uint32_t mine = e;
        if (i0 + stride < m) codes_of(g1, i0 + stride);
        g1 = g2;
        g2 = page_at(i0 + 3 * stride);
        to_l2(g2, i0 + 3 * stride);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
            for (int o = 4; o < 32; o *= 2) best[k] = fmaxf(best[k], __shfl_xor_sync(0xFFFFFFFFu, best[k], o));
            const uint32_t ek = __shfl_sync(0xFFFFFFFFu, mine, 4 * (2 * pair + k));
            const int i = i0 + 2 * pair + k;
            // (2^-20 of the score: below 2^128 for every exponent, and down to 2^-146, still exactly)
            if (quad == k && i < m)
                first_keys[i] = ek == 255 ? 0xFF800000u : ordered(best[k] * 0x1p-20f * __uint_as_float(ek << 23));
        }
    }
    if (astray && h == 0) atomicOr(p.c.err, kCacheErrPage);
    if (blocks > 1) cluster.sync();
    else __syncthreads();
    if (rank) return;
    select_largest<kSelectThreads>(m, K, sh.sel, [&](int i) { return keys[i]; },
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
    const int grid = (int)std::min<long long>((items + warps - 1) / warps, (long long)update_blocks(e4m3) * n_sm);
    auto go = [&](auto* f) { return launch_dependent(f, dim3((unsigned)grid), kUpdateThreads, 0, stream, p); };
    if (p.c.d == 64) return e4m3 ? go(update_kernel<64, true>) : go(update_kernel<64, false>);
    return e4m3 ? go(update_kernel<128, true>) : go(update_kernel<128, false>);
}

cudaError_t launch_bounds_select(const SelectParams& p, int n_sm, cudaStream_t stream) {
    const int units = p.B * p.Hkv;
    int cluster = 1;  // more blocks while they would be idle and a block has several rounds of pages
    while (cluster < 8 && 2LL * cluster * units <= 2LL * n_sm && p.t.max_pages > cluster * 24 * kSelectWarps) cluster *= 2;
    const int smem = 4 * p.t.max_pages;
    auto go = [&](auto* f) {
        const cudaError_t e = smem_opt_in(reinterpret_cast<const void*>(f), 4 * kSelectMostPages);
        return e != cudaSuccess ? e : launch_cluster(f, units * cluster, cluster, kSelectThreads, smem, stream, p);
    };
    if (p.c.d == 64) return p.rows <= 16 ? go(select_kernel<64, 1>) : go(select_kernel<64, 4>);
    return p.rows <= 16 ? go(select_kernel<128, 1>) : go(select_kernel<128, 4>);
}

}  // namespace attn
