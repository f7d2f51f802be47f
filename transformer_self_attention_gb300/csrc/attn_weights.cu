// The attention weight that each cached position receives, and eviction by it.
//
// Accumulation, after a decode step whose logarithms of sums are at hand: for every position j and kv head,
//     W_j <- decay * W_j + sum over the head's rows i that see j of exp(scale q_i . k_j - LSE_i)
// (positions of the step itself begin at 0).  Bound by memory: the keys are read once, W is read and written; 2 d flops a
// row and element.  The split of the work over the CTAs is the decode's (paged.h), by blocks of 16 positions; inside a
// stretch they go to the warps in turn, and nothing is shared, so that a position's sum has one owner and one order.
// Each warp has a ring of its own in shared memory and fills it itself: a TMA box of 16 keys, their W and exponents, a few
// blocks ahead.  The products are m16n8k16 with the rows as the first operand.  A lane's piece of a key is 16 bytes as they
// lie in memory: the order of a row's elements in the sum is free, so that the queries are permuted to match (a
// lane's 16 bytes are the elements that it would hold of two steps, or four of codes).
//
// Eviction: of each sequence and kv head the `keep` positions of largest W among all but the last `recent`, and those,
// moved to the front in their order.  One block finds the chosen positions of a head (select.h); then rows are
// copied, 16 bytes a lane at a time.  Into other pages all rows are copied at once, eight loads under way; in place a
// block takes a head's keys or values from front to back: a row moves forward or stays, so that what a store
// overwrites has been read as long as the rows before it have.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "device_once.h"
#include "paged_device.h"
#include "select.h"

namespace attn {

using namespace ptx;

namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kKeys = 16;  // of a block
constexpr PagedShape kShape{kKeys, 8, 32};

template <bool F16>
__device__ __forceinline__ void mma16(float (&c)[4], const uint4& a, uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// Four E4M3 codes as two pairs of fp16 numbers (exact).
__device__ __forceinline__ void widen_e4m3(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"((uint16_t)w));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"((uint16_t)(w >> 16)));
}
// Two bf16 numbers times a power of two, as fp16 numbers.
__device__ __forceinline__ uint32_t to_f16(uint32_t w, float scale) {
    uint32_t y;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(__uint_as_float(w & 0xFFFF0000u) * scale), "f"(__uint_as_float(w << 16) * scale));
    return y;
}

// A place of a warp's ring: 16 positions' keys (swizzled by the TMA load), their W, and (E4M3) their exponents.
template <int D, bool E4M3>
struct Place {
    static constexpr int kRow = D * (E4M3 ? 1 : 2);        // bytes of a key
    static constexpr int kSwizzled = kRow < 128 ? kRow : 128;  // a row comes in parts of so many bytes
    static constexpr int kBytes = kKeys * kRow;
    static constexpr int kSide = 128, kOffE = 64;          // beside the rings: W, and the exponents behind them
    static_assert(kBytes % 1024 == 0, "swizzled by address");
};
template <int D, bool E4M3, int RT>
struct WeighCfg {
    using P = Place<D, E4M3>;
    static constexpr int kCtas = RT == 4 ? 1 : 2;
    static constexpr int kFrag = RT == 1 ? 0 : RT * (D / 16) * 512;  // the queries as the products take them
    static constexpr int kRoom = (kCtas == 2 ? 113 : 225) * 1024 - 1024 - 6 * 1024 - kFrag;
    static constexpr int kFit = kRoom / (kWarps * (P::kBytes + P::kSide));
    static constexpr int kStages = kFit < 6 ? kFit : 6;
    static constexpr int kOffSide = kStages * kWarps * P::kBytes, kOffFrag = kOffSide + kStages * kWarps * P::kSide;
    static constexpr int kSmem = 1024 + kOffFrag + kFrag;
    static_assert(kStages >= 2, "a ring");
};

template <int D, bool E4M3, int RT>
__global__ void __launch_bounds__(kThreads, (WeighCfg<D, E4M3, RT>::kCtas)) weigh_kernel(const __grid_constant__ WeighParams wp) {
    using C = WeighCfg<D, E4M3, RT>;
    using P = Place<D, E4M3>;
    const PagedParams& p = wp.g;
    constexpr int kSteps = D / 16;  // products of a key tile and row tile
    constexpr int kStages = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    __shared__ unsigned cost[kPagedMaxBatch + 4];
    __shared__ unsigned scan[kWarps];
    __shared__ unsigned long long full[kWarps][kStages];
    __shared__ int abort_;
    uint8_t* const smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint4* const frag = reinterpret_cast<uint4*>(smem + C::kOffFrag);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int quad = lane / 4, pair = lane % 4, Hkv = p.Hkv, S_q = p.S_q;
    const uint32_t ring = smem_u32(smem) + warp * kStages * P::kBytes;
    const uint32_t sides = smem_u32(smem) + C::kOffSide + warp * kStages * P::kSide;
    if (lane == 0)
        for (int i = 0; i < kStages; ++i) mbar_init(smem_u32(&full[warp][i]), 1);
    if (tid == 0) {
        prefetch_tmap(&p.tm);
        abort_ = 0;
    }
    fence_barrier_init();
    wait_for_kernel_before();
    int busy;
    const unsigned W = paged_prefix<kKeys, kThreads>(p, kShape, cost, scan, busy) * p.units;
    const PagedCuts cuts(W, busy * p.units, gridDim.x, kShape);
    let_kernel_behind_in();
    if (blockIdx.x >= cuts.C || W == 0) return;
    const Watch watch{&abort_, p.c.err, p.watchdog_ns};
    Walk w = paged_begin(p, cuts, cost);
    const float log2e = 1.4426950408889634f;
    int filled = 0, taken = 0;  // blocks of the warp so far
    bool ok = true;
    while (w.at < w.end) {
        paged_open<kKeys>(p, kShape, cost, w);
        if (w.g0 >= w.g1) continue;
        const int len = w.len;
        const int n_mine = ok ? (w.g1 - w.g0 - warp + kWarps - 1) / kWarps : 0;
        // positions that a row of the sequence sees begin here; older blocks only fade
        const int seen = wp.window < 0 ? 0 : max(0, len - S_q - wp.window);
        auto block_of = [&](int i) { return w.lo + w.g0 + warp + i * kWarps; };
        // ---- loads, the warp's own, kStages blocks ahead.  Lane j has the page of the batch's j-th block, and the place in it.
        int pages = -1, slots = 0;       // of the blocks that are loaded next
        int pages_now = -1, slots_now = 0;  // of those that are worked on
        auto look_up = [&](int i0) {
            pages = -1;
            if (i0 + lane < n_mine) {
                const unsigned pos = (unsigned)block_of(i0 + lane) * kKeys, index = pos / (unsigned)p.c.page;
                slots = (int)(pos - index * p.c.page);
                pages = p.t.pages[w.b * p.t.stride + index];
                if (pages < 0 || pages >= p.c.n_pages) {
                    atomicOr(p.c.err, kCacheErrPage);
                    pages = -1;
                }
            }
        };
        auto load = [&](int i) {  // block i of the stretch; the batch of its page is the current one
            const int page = max(0, __shfl_sync(0xFFFFFFFFu, pages, i % 32)), slot = __shfl_sync(0xFFFFFFFFu, slots, i % 32);
            if (lane == 0) {
                const int st = filled % kStages;
                const uint32_t dst = ring + st * P::kBytes, side = sides + st * P::kSide, bar = smem_u32(&full[warp][st]);
                const long long unit = (long long)page * Hkv + w.h;
                const bool keys = block_of(i) * kKeys + kKeys > seen;
                mbar_arrive_expect_tx(bar, 4 * kKeys + (keys ? kKeys * P::kRow + (E4M3 ? 16 : 0) : 0));
                bulk_load(side, wp.w + unit * p.c.page + slot, 4 * kKeys, bar);
                if (keys) {
                    if constexpr (E4M3) {
                        asm volatile(
                            "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                            " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
                            "l"(reinterpret_cast<uint64_t>(&p.tm)), "r"(0), "r"(slot), "r"(0), "r"((int)unit), "r"(bar)
                            : "memory");
                        bulk_load(side + P::kOffE, p.c.scales + (unit * (p.c.page / 16) + slot / 16) * 32, 16, bar);
                    } else {
                        asm volatile(
                            "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                            " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
                            "l"(reinterpret_cast<uint64_t>(&p.tm)), "r"(0), "r"(slot), "r"(0), "r"(0), "r"((int)unit), "r"(bar)
                            : "memory");
                    }
                }
            }
            ++filled;
        };
        look_up(0);
        pages_now = pages;
        slots_now = slots;
        for (int i = 0; i < min(kStages - 1, n_mine); ++i) load(i);

        // ---- the queries.  A step's words of row tile r: rows quad and quad + 8 alternate, 4 of the lane's 8 (bf16) or 16
        // (E4M3) neighbouring elements
        auto query_words = [&](int r, int ks) {
            const uint16_t* q = reinterpret_cast<const uint16_t*>(p.q) + ((long long)w.b * Hkv + w.h) * p.rows * D;
            const int ra = 16 * r + quad, rb = ra + 8;
            const int at = E4M3 ? (ks / 4) * 64 + 16 * pair + 4 * (ks % 4) : (ks / 2) * 32 + 8 * pair + 4 * (ks % 2);
            const uint2 zero = make_uint2(0, 0);
            const uint2 a = ra < p.rows ? *reinterpret_cast<const uint2*>(q + (long long)ra * D + at) : zero;
            const uint2 b = rb < p.rows ? *reinterpret_cast<const uint2*>(q + (long long)rb * D + at) : zero;
            return make_uint4(a.x, b.x, a.y, b.y);
        };
        // E4M3: codes are fp16 numbers in the products, and so are the queries, each row times a power of two that brings its
        // largest element to 2^14 .. 2^15 (elements below 2^-28 of that lose bits, 2^-39 of it at most); `up` undoes it
        float up[2 * RT];
        uint4 qf[RT == 1 ? kSteps : 1];
        if constexpr (RT > 1) __syncthreads();
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            uint4 q[kSteps];
#pragma unroll
            for (int ks = 0; ks < kSteps; ++ks) q[ks] = query_words(r, ks);
            if constexpr (E4M3) {
                uint32_t big[2] = {0, 0};  // as bits of bf16 numbers
#pragma unroll
                for (int ks = 0; ks < kSteps; ++ks) {
                    big[0] = __vmaxu2(big[0], __vmaxu2(q[ks].x & 0x7FFF7FFFu, q[ks].z & 0x7FFF7FFFu));
                    big[1] = __vmaxu2(big[1], __vmaxu2(q[ks].y & 0x7FFF7FFFu, q[ks].w & 0x7FFF7FFFu));
                }
                float down[2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    uint32_t t = max(big[x] & 0xFFFFu, big[x] >> 16);
                    t = max(t, __shfl_xor_sync(0xFFFFFFFFu, t, 1));
                    t = max(t, __shfl_xor_sync(0xFFFFFFFFu, t, 2));
                    // exponent field e: the row is below 2^(e - 126), so below 2^15 times 2^(141 - e).  A row below 2^-100
                    // is taken as zeros in part; one with an infinity or a NaN becomes NaN.
                    const int e = max((int)(t >> 7), 27);
                    down[x] = e == 255 ? __int_as_float(0x7FFFFFFF) : __uint_as_float((uint32_t)min(268 - e, 254) << 23);
                    up[2 * r + x] = __uint_as_float((uint32_t)max(e - 14, 0) << 23);
                    if (e == 255) up[2 * r + x] = 1.f;
                }
#pragma unroll
                for (int ks = 0; ks < kSteps; ++ks)
                    q[ks] = make_uint4(to_f16(q[ks].x, down[0]), to_f16(q[ks].y, down[1]), to_f16(q[ks].z, down[0]),
                                       to_f16(q[ks].w, down[1]));
            }
#pragma unroll
            for (int ks = 0; ks < kSteps; ++ks) {
                if constexpr (RT == 1) qf[ks] = q[ks];
                else if ((r * kSteps + ks) % kWarps == warp) frag[(r * kSteps + ks) * 32 + lane] = q[ks];
            }
        }
        if constexpr (RT > 1) __syncthreads();
        // rows quad and quad + 8 of every row tile: what is taken off the exponent, and the positions they see
        float lse[2 * RT];
        int last[2 * RT], first_seen[2 * RT];
        bool dead = false;  // a row of the sequence has no weights
#pragma unroll
        for (int r = 0; r < 2 * RT; ++r) {
            const int row = 16 * (r / 2) + 8 * (r % 2) + quad;
            const float x = row < p.rows ? wp.lse[((long long)w.b * Hkv + w.h) * p.rows + row] : 0.f;
            const int t = len - S_q + row % S_q;
            const bool none = x == __int_as_float(0xFF800000);
            lse[r] = x * log2e;
            if constexpr (E4M3) up[r] *= p.scale_log2;
            last[r] = none || row >= p.rows ? -1 : p.causal ? t : len - 1;
            first_seen[r] = wp.window < 0 ? 0 : max(0, t - wp.window);
            dead |= none;
        }
        dead = __any_sync(0xFFFFFFFFu, dead);
        const int all_to = p.causal ? len - S_q + 1 : len;
        const int all_from = wp.window < 0 ? 0 : max(0, len - 1 - wp.window);
        // the lane's position of a block, after the sums over the rows: key 8 (lane / 16) + 2 pair + (lane / 8) % 2
        const int mine = 8 * (lane / 16) + 2 * pair + (lane / 8) % 2;

        for (int i = 0; i < n_mine && ok; ++i) {
            // the place that the block before left is filled again
            const int ahead = i + kStages - 1;
            if (ahead < n_mine) {
                if (ahead % 32 == 0) {
                    __syncwarp();
                    look_up(ahead);
                }
                load(ahead);
            }
            if (i % 32 == 0 && i > 0) {  // (kStages <= 32: the batch that is loaded from holds this block's page too)
                pages_now = pages;
                slots_now = slots;
            }
            const int st = taken % kStages;
            const uint32_t buf = ring + st * P::kBytes, side = sides + st * P::kSide;
            ok = __all_sync(0xFFFFFFFFu, wait(smem_u32(&full[warp][st]), (taken / kStages) & 1, watch));
            if (!ok) break;
            const int pos = block_of(i) * kKeys;
            float sum[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
            if (pos + kKeys > seen) {
                // a lane's pieces of the keys quad and quad + 8, 16 bytes each
                uint4 k[2][P::kRow / 64];
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int l = 0; l < P::kRow / 64; ++l) {
                        const int row = quad + 8 * j, chunk = 4 * (l % (P::kSwizzled / 64)) + pair;
                        const int sw = P::kSwizzled == 128 ? chunk ^ (row & 7) : chunk ^ ((row >> 1) & 3);
                        k[j][l] = lds16(buf + (l / (P::kSwizzled / 64)) * kKeys * P::kSwizzled + row * P::kSwizzled + 16 * sw);
                    }
                float factor[2][2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint32_t e = 0;  // of the keys whose products the lane gets: 2 pair and 2 pair + 1 of either tile
                    if (E4M3)
                        asm volatile("ld.shared.u16 %0, [%1];" : "=r"(e) : "r"(side + P::kOffE + 8 * j + 2 * pair) : "memory");
#pragma unroll
                    for (int c = 0; c < 2; ++c)  // (255: NaN codes beside it)
                        factor[j][c] = __uint_as_float(max((e >> 8 * c & 0xFF) << 23, 0x00400000u));
                }
                const bool check = dead || pos < all_from || pos + kKeys > all_to;
                uint32_t kb[2][2 * kSteps];  // the keys as 16-bit numbers
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int l = 0; l < P::kRow / 64; ++l) {
                        const uint32_t v[4] = {k[j][l].x, k[j][l].y, k[j][l].z, k[j][l].w};
                        if constexpr (E4M3) {
#pragma unroll
                            for (int x = 0; x < 4; ++x) widen_e4m3(v[x], kb[j][8 * l + 2 * x], kb[j][8 * l + 2 * x + 1]);
                        } else {
#pragma unroll
                            for (int x = 0; x < 4; ++x) kb[j][4 * l + x] = v[x];
                        }
                    }
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    float s[2][2][4];  // two chains a tile
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int c = 0; c < 4; ++c) s[j][0][c] = s[j][1][c] = 0.f;
#pragma unroll
                    for (int ks = 0; ks < kSteps; ++ks) {
                        const uint4 a = RT == 1 ? qf[RT == 1 ? ks : 0] : frag[(r * kSteps + ks) * 32 + lane];
#pragma unroll
                        for (int j = 0; j < 2; ++j) mma16<E4M3>(s[j][ks % 2], a, kb[j][2 * ks], kb[j][2 * ks + 1]);
                    }
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const int row = 2 * r + c / 2;
                            const float scale = E4M3 ? factor[j][c % 2] * up[row] : p.scale_log2;
                            float y = ex2(fmaf(s[j][0][c] + s[j][1][c], scale, -lse[row]));
                            if (check) {
                                const int at = pos + 8 * j + 2 * pair + c % 2;
                                if (at > last[row] || at < first_seen[row]) y = 0.f;
                            } else if (16 * (row / 2) + 8 * (row % 2) + quad >= p.rows) {
                                y = 0.f;
                            }
                            sum[j][c % 2] += y;
                        }
                }
            }
            // over the rows' lanes, half of the values given away with each step: tile, then key, then both halves
            float v[2];
            {
                const bool up = lane & 16;
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    v[c] = (up ? sum[1][c] : sum[0][c]) + __shfl_xor_sync(0xFFFFFFFFu, up ? sum[0][c] : sum[1][c], 16);
            }
            const bool odd = lane & 8;
            float total = (odd ? v[1] : v[0]) + __shfl_xor_sync(0xFFFFFFFFu, odd ? v[0] : v[1], 8);
            total += __shfl_xor_sync(0xFFFFFFFFu, total, 4);
            float old;
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(old) : "r"(side + 4 * mine) : "memory");
            if (pos + mine >= len - S_q) old = 0.f;  // (whatever it holds)
            const int page = __shfl_sync(0xFFFFFFFFu, pages_now, i % 32), slot = __shfl_sync(0xFFFFFFFFu, slots_now, i % 32);
            if ((lane & 4) == 0 && pos + mine < len && page >= 0)
                wp.w[((long long)page * Hkv + w.h) * p.c.page + slot + mine] = fmaf(wp.decay, old, total);
            ++taken;
            __syncwarp();  // the block is read: its place may be filled again
        }
    }
    // all warps meet behind their last copy; after a wait that ran out those on their way are waited for
    __syncthreads();
    if (abort_) drain();
}

// ---------------------------------------------------------------------------------------------- eviction
constexpr int kRankThreads = 1024;

__global__ void __launch_bounds__(kRankThreads, 1) rank_kernel(const __grid_constant__ EvictParams p) {
    __shared__ SelectShared<kRankThreads> sh;
    extern __shared__ __align__(16) uint32_t keys[];
    const int tid = threadIdx.x, unit = blockIdx.x, b = unit / p.c.Hkv, h = unit - b * p.c.Hkv, page = p.c.page;
    wait_for_kernel_before();
    let_kernel_behind_in();
    int n = p.t.len[b];
    if (n < 0 || n > p.t.max_pages * page) {
        if (tid == 0 && h == 0) atomicOr(p.c.err, kCacheErrPosition);
        n = 0;
    }
    const int stay = p.keep + p.recent, left = min(n, stay), old = max(0, n - p.recent);
    int* kept = p.kept + (long long)unit * stay;
    if (h == 0 && tid == 0) p.out_len[b] = left;
    const int* row = p.t.pages + b * p.t.stride;
    for (int i = tid; i < stay; i += kRankThreads) {
        if (i >= left) kept[i] = -1;
        else if (n <= stay) kept[i] = i;
        else if (i >= p.keep) kept[i] = old + i - p.keep;
    }
    if (n <= stay) return;
    const int Hkv = p.c.Hkv;
    bool astray = false;
    auto page_of = [&](int i, int& slot) {
        const int index = (unsigned)i / (unsigned)page;
        slot = i - index * page;
        return row[index];
    };
    auto weight_in = [&](int g, int slot) {  // (a page out of range: as light as can be)
        const bool ok = g >= 0 && g < p.c.n_pages;
        astray |= !ok;
        return ok ? ordered(p.w[((long long)g * Hkv + h) * page + slot]) : 0u;
    };
    auto emit = [&](int place, int i) { kept[place] = i; };
    if (old <= p.cached) {
        // four neighbours to a thread (they are in one page: its size is a multiple of 16), pages, then weights, at once
        constexpr int kAhead = 4;
        for (int i0 = 4 * tid; i0 < old; i0 += 4 * kAhead * kRankThreads) {
            int g[kAhead], slot[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) g[j] = page_of(min(i0 + 4 * j * kRankThreads, (old - 1) & ~3), slot[j]);
            float4 v[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const bool ok = g[j] >= 0 && g[j] < p.c.n_pages;
                astray |= !ok;
                v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (ok) v[j] = *reinterpret_cast<const float4*>(p.w + ((long long)g[j] * Hkv + h) * page + slot[j]);
                else slot[j] = -1;  // as light as can be
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int i = i0 + 4 * j * kRankThreads;  // (room for the last four: the places' number is rounded up)
                if (i < old)
                    *reinterpret_cast<uint4*>(&keys[i]) =
                        slot[j] < 0 ? make_uint4(0, 0, 0, 0)
                                    : make_uint4(ordered(v[j].x), ordered(v[j].y), ordered(v[j].z), ordered(v[j].w));
            }
        }
        __syncthreads();
        select_largest<kRankThreads>(old, p.keep, sh, [&](int i) { return keys[i]; }, emit);
    } else {
        select_largest<kRankThreads>(old, p.keep, sh, [&](int i) {
            int slot;
            const int g = page_of(i, slot);
            return weight_in(g, slot);
        }, emit);
    }
    if (astray) atomicOr(p.c.err, kCacheErrPage);
}

// A row's place in memory: [page][head][keys, values][slot].
struct RowAt {
    int page, slot;
};
__device__ __forceinline__ RowAt row_at(const EvictParams& p, const int* row, int i) {
    const int index = (unsigned)i / (unsigned)p.c.page;
    RowAt r{row[index], i - index * p.c.page};
    if (r.page < 0 || r.page >= p.c.n_pages) {
        atomicOr(p.c.err, kCacheErrPage);
        r.page = -1;
    }
    return r;
}
__device__ __forceinline__ long long scale_at(const EvictParams& p, RowAt r, int h) {
    return (((long long)r.page * p.c.Hkv + h) * (p.c.page / 16) + r.slot / 16) * 32 + r.slot % 16;
}
__device__ __forceinline__ long long weight_at(const EvictParams& p, RowAt r, int h) {
    return ((long long)r.page * p.c.Hkv + h) * p.c.page + r.slot;
}

// Into other pages: a warp takes 32 rows of one head after another (eight where there are too few for all warps), a lane
// looks up one row, and all lanes copy them, 512 bytes at a time, eight loads under way; the next rows are looked up
// meanwhile.
constexpr int kMoveBlocks = 4;  // a multiprocessor, all at once
template <int ROWB>  // bytes of a key
__global__ void __launch_bounds__(kThreads, kMoveBlocks) move_kernel(const __grid_constant__ EvictParams p, int groups, int per) {
    constexpr int kLanes = ROWB / 16, kAtOnce = 32 / kLanes, kAhead = 8;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    wait_for_kernel_before();
    let_kernel_behind_in();
    const int items = p.B * p.c.Hkv * groups, stay = p.keep + p.recent, step = gridDim.x * kWarps;
    const long long side = (long long)p.c.page * ROWB;  // from a key to its value
    const int sub = lane / kLanes, off = 16 * (lane % kLanes);
    auto kept_of = [&](int item) {
        const int unit = item / groups, i = (item - unit * groups) * per + lane;
        return item < items && lane < per && i < stay ? p.kept[(long long)unit * stay + i] : -1;
    };
    struct Where {
        RowAt src, dst;
        int from;
    };
    auto look_up = [&](int item, int from) {
        Where w{{-1, 0}, {-1, 0}, from};
        if (from >= 0) {
            const int unit = item / groups, i = (item - unit * groups) * per + lane, b = unit / p.c.Hkv;
            w.src = row_at(p, p.t.pages + b * p.t.stride, from);
            w.dst = row_at(p, p.to + b * p.to_stride, i);
        }
        return w;
    };
    int item = blockIdx.x * kWarps + warp;
    Where now = look_up(item, kept_of(item));
    for (; item < items; item += step) {
        const int next_from = kept_of(item + step), h = item / groups % p.c.Hkv;
        Where next{{-1, 0}, {-1, 0}, -1};
        const bool ok = now.src.page >= 0 && now.dst.page >= 0;
        if (ok) {
            p.w[weight_at(p, now.dst, h)] = p.w[weight_at(p, now.src, h)];
            if (p.c.scales) {
                const uint8_t* s = p.c.scales + scale_at(p, now.src, h);
                uint8_t* d = p.c.scales + scale_at(p, now.dst, h);
                d[0] = s[0];
                d[16] = s[16];
            }
        }
        const int n = __popc(__ballot_sync(0xFFFFFFFFu, now.from >= 0));  // (the first lanes)
        // where the lane's row begins; -1: it is not moved
        const long long s0 = ok ? (((long long)now.src.page * p.c.Hkv + h) * 2 * p.c.page + now.src.slot) * ROWB : -1;
        const long long d0 = (((long long)now.dst.page * p.c.Hkv + h) * 2 * p.c.page + now.dst.slot) * ROWB;
        bool looked = false;
        for (int r = 0; r < 2 * n; r += kAhead * kAtOnce) {  // rows: the keys, then the values, of row r / 2
            uint4 v[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int x = r + k * kAtOnce + sub;
                const long long s = __shfl_sync(0xFFFFFFFFu, s0, min(x / 2, 31));
                if (s >= 0 && x < 2 * n) v[k] = *reinterpret_cast<const uint4*>(p.c.pages + s + (x % 2) * side + off);
            }
            if (!looked) next = look_up(item + step, next_from);
            looked = true;
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int x = r + k * kAtOnce + sub;
                const long long s = __shfl_sync(0xFFFFFFFFu, s0, min(x / 2, 31)), d = __shfl_sync(0xFFFFFFFFu, d0, min(x / 2, 31));
                if (s >= 0 && x < 2 * n) *reinterpret_cast<uint4*>(p.c.pages + d + (x % 2) * side + off) = v[k];
            }
        }
        if (!looked) next = look_up(item + step, next_from);
        now = next;
    }
}

// In place: a block takes SLICE bytes of each of a head's keys or values (blockIdx.y) from front to back, kRows rows a
// round.  A round's loads are all done (the barrier) before its first store; the next round's may come before them too:
// rows are read at their place or behind it.  Slices of 64 bytes make more blocks and rounds of more rows: 186 us for 64 heads of
// 32K positions of 256 bytes cut to 8448, 294 with whole rows; with blocks enough whole rows are better (512 heads of 2K cut to 768:
// 110 us, 124 with slices).
constexpr int kPlaceThreads = 512;
template <int ROWB, int SLICE>
__global__ void __launch_bounds__(kPlaceThreads) move_in_place_kernel(const __grid_constant__ EvictParams p) {
    constexpr int kLanes = SLICE / 16, kEach = 4, kStep = kPlaceThreads / kLanes, kRows = kEach * kStep;
    const int tid = threadIdx.x, unit = blockIdx.x, b = unit / p.c.Hkv, h = unit - b * p.c.Hkv, kv = blockIdx.y % 2;
    wait_for_kernel_before();
    let_kernel_behind_in();
    const int stay = p.keep + p.recent;
    const int* row = p.t.pages + b * p.t.stride;
    const int* kept = p.kept + (long long)unit * stay;
    const int sub = tid / kLanes, off = blockIdx.y / 2 * SLICE + 16 * (tid % kLanes);
    int n = p.t.len[b];
    if (n <= stay || n > p.t.max_pages * p.c.page) return;  // every row stays where it is
    for (int r0 = 0; r0 < stay; r0 += kRows) {
        uint4 v[kEach];
        float weight[kEach];
        uint8_t e[kEach];
        RowAt dst[kEach];
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int i = r0 + k * kStep + sub;
            dst[k].page = -1;
            if (i >= stay) continue;
            const int from = kept[i];
            if (from <= i) continue;  // (it stays; nothing moves back, and -1 is no place)
            const RowAt src = row_at(p, row, from);
            dst[k] = row_at(p, row, i);
            if (src.page < 0) dst[k].page = -1;
            if (dst[k].page < 0) continue;
            v[k] = *reinterpret_cast<const uint4*>(
                p.c.pages + ((((long long)src.page * p.c.Hkv + h) * 2 + kv) * p.c.page + src.slot) * ROWB + off);
            if (off == 0) {
                if (kv == 0) weight[k] = p.w[weight_at(p, src, h)];
                if (p.c.scales) e[k] = p.c.scales[scale_at(p, src, h) + 16 * kv];
            }
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            if (dst[k].page < 0) continue;
            *reinterpret_cast<uint4*>(
                p.c.pages + ((((long long)dst[k].page * p.c.Hkv + h) * 2 + kv) * p.c.page + dst[k].slot) * ROWB + off) = v[k];
            if (off == 0) {
                if (kv == 0) p.w[weight_at(p, dst[k], h)] = weight[k];
                if (p.c.scales) p.c.scales[scale_at(p, dst[k], h) + 16 * kv] = e[k];
            }
        }
    }
}

}  // namespace

cudaError_t launch_weigh(const WeighParams& p, bool e4m3, int n_sm, cudaStream_t stream) {
    const int tiles = (p.g.rows + 15) / 16, rt = tiles <= 1 ? 1 : tiles <= 2 ? 2 : 4;
    auto go = [&](auto* f, int smem, int ctas) {
        const cudaError_t e = smem_opt_in(reinterpret_cast<const void*>(f), smem);
        return e != cudaSuccess ? e : launch_dependent(f, dim3((unsigned)(n_sm * ctas)), kThreads, smem, stream, p);
    };
    auto of_rows = [&](auto d, auto type) {
        constexpr int D = decltype(d)::value;
        constexpr bool E = decltype(type)::value;
        auto with = [&](auto t) {
            using C = WeighCfg<D, E, decltype(t)::value>;
            return go(weigh_kernel<D, E, decltype(t)::value>, C::kSmem, C::kCtas);
        };
        return rt == 1 ? with(std::integral_constant<int, 1>{})
                       : rt == 2 ? with(std::integral_constant<int, 2>{}) : with(std::integral_constant<int, 4>{});
    };
    using D64 = std::integral_constant<int, 64>;
    using D128 = std::integral_constant<int, 128>;
    if (p.g.c.d == 64) return e4m3 ? of_rows(D64{}, std::true_type{}) : of_rows(D64{}, std::false_type{});
    return e4m3 ? of_rows(D128{}, std::true_type{}) : of_rows(D128{}, std::false_type{});
}

cudaError_t launch_evict(EvictParams p, bool e4m3, int n_sm, cudaStream_t stream) {
    const int units = p.B * p.c.Hkv, stay = p.keep + p.recent;
    p.cached = (int)std::min<long long>((long long)p.t.max_pages * p.c.page, kEvictCached);
    cudaError_t e = smem_opt_in(reinterpret_cast<const void*>(&rank_kernel), 4 * kEvictCached);
    if (e != cudaSuccess) return e;
    e = launch_dependent(rank_kernel, dim3((unsigned)units), kRankThreads, 4 * p.cached, stream, p);
    if (e != cudaSuccess) return e;
    const int rowb = p.c.d * (e4m3 ? 1 : 2);
    if (p.in_place) {
        const bool whole = 2 * units >= 4 * n_sm;
        auto go = [&](auto width) {
            constexpr int W = decltype(width)::value;
            return whole ? launch_dependent(move_in_place_kernel<W, W>, dim3((unsigned)units, 2), kPlaceThreads, 0, stream, p)
                         : launch_dependent(move_in_place_kernel<W, 64>, dim3((unsigned)units, 2 * W / 64), kPlaceThreads, 0, stream, p);
        };
        return rowb == 64 ? go(std::integral_constant<int, 64>{})
                          : rowb == 128 ? go(std::integral_constant<int, 128>{}) : go(std::integral_constant<int, 256>{});
    }
    const int rows = (int)std::min<long long>(stay, (long long)p.t.max_pages * p.c.page), most = kMoveBlocks * n_sm;
    const int per = (long long)units * rows >= 32LL * kWarps * most ? 32 : 8, groups = (rows + per - 1) / per;
    const dim3 grid((unsigned)std::min<long long>(((long long)units * groups + kWarps - 1) / kWarps, most));
    auto go = [&](auto* f) { return launch_dependent(f, grid, kThreads, 0, stream, p, groups, per); };
    return rowb == 64 ? go(move_kernel<64>) : rowb == 128 ? go(move_kernel<128>) : go(move_kernel<256>);
}

}  // namespace attn
