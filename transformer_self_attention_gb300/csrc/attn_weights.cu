// The attention weight that each cached position receives, and eviction by it.
//
// Accumulation, after a decode step whose logarithms of sums are at hand: for every position j and kv head,
//     W_j <- decay * W_j + sum over the head's rows i that see j of exp(scale q_i . k_j - LSE_i)
// (positions of the step itself begin at 0).  Bound by memory: the keys are read once, W is read and written; 2 d flops a
// row and element.  The split of the work over the CTAs is the decode's (paged.h), by blocks of 16 positions; inside a
// stretch they go to the warps in turn, and nothing is shared, so that a position's sum has one owner and one order.
// The products are m16n8k16 with the rows as the first operand.  A lane's piece of a key is 16 bytes as they lie in
// memory, loaded to registers without a detour by shared memory: the order of a row's elements in the sum is free, so that
// the queries are permuted to match (a lane's 16 bytes are the elements that it would hold of two steps).
//
// Eviction: of each sequence and kv head the `keep` positions of largest W among all but the last `recent`, and those,
// moved to the front in their order.  One block finds the chosen positions of a head (select.h); then rows are
// copied, two loads and stores of 16 bytes a lane and row.  Into other pages all rows are copied at once; in place a
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

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Four E4M3 codes as two pairs of bf16 numbers (exact).
__device__ __forceinline__ void widen_e4m3(uint32_t w, uint32_t& lo, uint32_t& hi) {
    uint32_t h0, h1;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h0) : "h"((uint16_t)w));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h1) : "h"((uint16_t)(w >> 16)));
    float a, b;
    asm("{.reg .f16 x, y; mov.b32 {x, y}, %2; cvt.f32.f16 %0, x; cvt.f32.f16 %1, y;}" : "=f"(a), "=f"(b) : "r"(h0));
    lo = pack_bf16x2(a, b);
    asm("{.reg .f16 x, y; mov.b32 {x, y}, %2; cvt.f32.f16 %0, x; cvt.f32.f16 %1, y;}" : "=f"(a), "=f"(b) : "r"(h1));
    hi = pack_bf16x2(a, b);
}

// A lane's loads of one block: its pieces of the keys quad and quad + 8, and (E4M3) their exponents.
template <int D, bool E4M3>
struct Piece {
    static constexpr int kLoads = D * (E4M3 ? 1 : 2) / 64;  // of a key
    uint4 k[2][kLoads];
    uint32_t e[2];
    float old;  // W of the lane's position
};

template <int D, bool E4M3, int RT>
__global__ void __launch_bounds__(kThreads, RT == 1 ? 2 : 1) weigh_kernel(const __grid_constant__ WeighParams wp) {
    const PagedParams& p = wp.g;
    constexpr int kSteps = D / 16;  // products of a key tile and row tile
    __shared__ unsigned cost[kPagedMaxBatch + 4];
    __shared__ unsigned scan[kWarps];
    __shared__ uint4 frag[RT == 1 ? 1 : RT * kSteps * 32];  // the queries as the products take them, a step's four words
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int quad = lane / 4, pair = lane % 4, Hkv = p.Hkv, S_q = p.S_q;
    wait_for_kernel_before();
    int busy;
    const unsigned W = paged_prefix<kKeys, kThreads>(p, kShape, cost, scan, busy) * p.units;
    const PagedCuts cuts(W, busy * p.units, gridDim.x, kShape);
    let_kernel_behind_in();
    if (blockIdx.x >= cuts.C || W == 0) return;
    Walk w = paged_begin(p, cuts, cost);
    const float log2e = 1.4426950408889634f;
    while (w.at < w.end) {
        paged_open<kKeys>(p, kShape, cost, w);
        if (w.g0 >= w.g1) continue;
        const int len = w.len;
        // a step's words of row tile r: rows quad and quad + 8 alternate
        auto query_words = [&](int r, int ks) {
            const uint16_t* q = reinterpret_cast<const uint16_t*>(p.q) + ((long long)w.b * Hkv + w.h) * p.rows * D;
            const int ra = 16 * r + quad, rb = ra + 8;
            // element of the step's first word: 4 of the lane's 8 (bf16) or 16 (E4M3) neighbouring elements
            const int at = E4M3 ? (ks / 4) * 64 + 16 * pair + 4 * (ks % 4) : (ks / 2) * 32 + 8 * pair + 4 * (ks % 2);
            const uint2 zero = make_uint2(0, 0);
            const uint2 a = ra < p.rows ? *reinterpret_cast<const uint2*>(q + (long long)ra * D + at) : zero;
            const uint2 b = rb < p.rows ? *reinterpret_cast<const uint2*>(q + (long long)rb * D + at) : zero;
            return make_uint4(a.x, b.x, a.y, b.y);
        };
        uint4 qf[RT == 1 ? kSteps : 1];
        if constexpr (RT == 1) {
#pragma unroll
            for (int ks = 0; ks < kSteps; ++ks) qf[ks] = query_words(0, ks);
        } else {
            __syncthreads();
            for (int i = warp; i < RT * kSteps; i += kWarps) frag[i * 32 + lane] = query_words(i / kSteps, i % kSteps);
            __syncthreads();
        }
        // rows quad and quad + 8 of every row tile: what is taken off the exponent, and the positions they see
        float lse[2 * RT];
        int last[2 * RT], first_seen[2 * RT];
#pragma unroll
        for (int r = 0; r < 2 * RT; ++r) {
            const int row = 16 * (r / 2) + 8 * (r % 2) + quad;
            const float x = row < p.rows ? wp.lse[((long long)w.b * Hkv + w.h) * p.rows + row] : 0.f;
            const int t = len - S_q + row % S_q;
            const bool dead = row >= p.rows || x == __int_as_float(0xFF800000);
            lse[r] = x * log2e;
            last[r] = dead ? -1 : p.causal ? t : len - 1;
            first_seen[r] = wp.window < 0 ? 0 : max(0, t - wp.window);
        }
        // positions that a row of the sequence sees
        const int seen = wp.window < 0 ? 0 : max(0, len - S_q - wp.window);
        const int all_to = p.causal ? len - S_q + 1 : len;
        const int all_from = wp.window < 0 ? 0 : max(0, len - 1 - wp.window);
        bool whole = true;  // no row of the lane is without weights
#pragma unroll
        for (int r = 0; r < 2 * RT; ++r) whole &= last[r] >= 0;
        whole = __all_sync(0xFFFFFFFFu, whole);
        // the lane's position of a block, after the sums over the rows: key 8 (lane / 16) + 2 pair + (lane / 8) % 2
        const int mine = 8 * (lane / 16) + 2 * pair + (lane / 8) % 2;
        int batch = 0;  // page numbers of the warp's next 32 blocks, a lane each
        const int n_mine = (w.g1 - w.g0 - warp + kWarps - 1) / kWarps;
        auto block_of = [&](int i) { return w.lo + w.g0 + warp + i * kWarps; };
        auto pages_from = [&](int i) {
            batch = 0;
            if (i + lane < n_mine) {
                const unsigned pos = (unsigned)block_of(i + lane) * kKeys;
                batch = p.t.pages[w.b * p.t.stride + pos / (unsigned)p.c.page];
                if (batch < 0 || batch >= p.c.n_pages) {
                    atomicOr(p.c.err, kCacheErrPage);
                    batch = -1;
                }
            }
        };
        using P = Piece<D, E4M3>;
        auto fetch = [&](int i, P& f) {
            if (i % 32 == 0) pages_from(i);
            if (i >= n_mine) return;
            const int page = __shfl_sync(0xFFFFFFFFu, batch, i % 32);
            const int pos = block_of(i) * kKeys, slot = pos % p.c.page;
            const long long unit = (long long)max(page, 0) * Hkv + w.h;
            if (pos + kKeys > seen) {  // (older positions only fade)
                const char* src = p.c.pages + (unit * 2 * p.c.page + slot + quad) * (D * (E4M3 ? 1 : 2)) + 16 * pair;
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int l = 0; l < P::kLoads; ++l)
                        f.k[j][l] = *reinterpret_cast<const uint4*>(src + 8 * j * (D * (E4M3 ? 1 : 2)) + 64 * l);
                if (E4M3) {  // of the keys whose products the lane gets: 2 pair and 2 pair + 1 of either tile
                    const uint8_t* sc = p.c.scales + (unit * (p.c.page / 16) + slot / 16) * 32 + 2 * pair;
                    f.e[0] = *reinterpret_cast<const uint16_t*>(sc);
                    f.e[1] = *reinterpret_cast<const uint16_t*>(sc + 8);
                }
            }
            f.old = pos + mine < len - S_q ? wp.w[unit * p.c.page + slot + mine] : 0.f;
        };
        auto take = [&](int i, const P& f) {
            const int page = __shfl_sync(0xFFFFFFFFu, batch, i % 32);
            const int pos = block_of(i) * kKeys, slot = pos % p.c.page;
            float sum[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
            if (pos + kKeys > seen) {
                const bool check = !whole || pos < all_from || pos + kKeys > all_to;
                float factor[2][2];
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const uint32_t e = f.e[j] >> 8 * c & 0xFF;  // (255: NaN codes beside it)
                        factor[j][c] = E4M3 ? p.scale_log2 * __uint_as_float(max(e << 23, 0x00400000u)) : p.scale_log2;
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
                        const uint4 a = RT == 1 ? qf[ks % (RT == 1 ? kSteps : 1)] : frag[(r * kSteps + ks) * 32 + lane];
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            uint32_t b0, b1;
                            if constexpr (E4M3) {
                                const uint4& v = f.k[j][ks / 4];
                                widen_e4m3(ks % 4 == 0 ? v.x : ks % 4 == 1 ? v.y : ks % 4 == 2 ? v.z : v.w, b0, b1);
                            } else {
                                const uint4& v = f.k[j][ks / 2];
                                b0 = ks % 2 ? v.z : v.x;
                                b1 = ks % 2 ? v.w : v.y;
                            }
                            mma_bf16(s[j][ks % 2], a.x, a.y, a.z, a.w, b0, b1);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const int row = 2 * r + c / 2;
                            const float x = s[j][0][c] + s[j][1][c];
                            float y = ex2(fmaf(x, factor[j][c % 2], -lse[row]));
                            if (check) {
                                const int at = pos + 8 * j + 2 * pair + c % 2;
                                if (at > last[row] || at < first_seen[row]) y = 0.f;
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
            if ((lane & 4) == 0 && pos + mine < len && page >= 0)
                wp.w[((long long)page * Hkv + w.h) * p.c.page + slot + mine] = fmaf(wp.decay, f.old, total);
        };
        P a, b;
        if (n_mine > 0) fetch(0, a);
        for (int i = 0; i < n_mine; i += 2) {
            // (the batch of page numbers changes at multiples of 32: the block before is through by then)
            fetch(i + 1, b);
            take(i, a);
            if (i + 1 < n_mine) take(i + 1, b);
            fetch(i + 2, a);
        }
    }
}

// ---------------------------------------------------------------------------------------------- eviction
constexpr int kRankThreads = 1024;

__global__ void __launch_bounds__(kRankThreads) rank_kernel(const __grid_constant__ EvictParams p) {
    __shared__ SelectShared<kRankThreads> sh;
    extern __shared__ uint32_t keys[];
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
    auto weight = [&](int i) {
        const int index = (unsigned)i / (unsigned)page;
        const int g = row[index];
        if (g < 0 || g >= p.c.n_pages) {
            atomicOr(p.c.err, kCacheErrPage);
            return 0u;
        }
        return ordered(p.w[((long long)g * p.c.Hkv + h) * page + (i - index * page)]);
    };
    auto emit = [&](int place, int i) { kept[place] = i; };
    if (old <= p.cached) {
        for (int i = tid; i < old; i += kRankThreads) keys[i] = weight(i);
        __syncthreads();
        select_largest<kRankThreads>(old, p.keep, sh, [&](int i) { return keys[i]; }, emit);
    } else {
        select_largest<kRankThreads>(old, p.keep, sh, weight, emit);
    }
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

// Into other pages: 32 rows of one head to a warp, a lane looks up one row, and all lanes copy them, 512 bytes at a time.
template <int ROWB>  // bytes of a key
__global__ void __launch_bounds__(kThreads) move_kernel(const __grid_constant__ EvictParams p, int groups) {
    constexpr int kLanes = ROWB / 16, kAtOnce = 32 / kLanes, kAhead = 8;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    wait_for_kernel_before();
    let_kernel_behind_in();
    const long long item = (long long)blockIdx.x * kWarps + warp;
    const int unit = (int)(item / groups), first = (int)(item - (long long)unit * groups) * 32;
    if (unit >= p.B * p.c.Hkv) return;
    const int b = unit / p.c.Hkv, h = unit - b * p.c.Hkv, stay = p.keep + p.recent;
    const int i = first + lane, from = i < stay ? p.kept[(long long)unit * stay + i] : -1;
    RowAt src{-1, 0}, dst{-1, 0};
    if (from >= 0) {
        src = row_at(p, p.t.pages + b * p.t.stride, from);
        dst = row_at(p, p.to + b * p.to_stride, i);
    }
    const bool ok = src.page >= 0 && dst.page >= 0;
    if (!__any_sync(0xFFFFFFFFu, ok)) return;
    if (ok) {
        p.w[weight_at(p, dst, h)] = p.w[weight_at(p, src, h)];
        if (p.c.scales) {
            const uint8_t* s = p.c.scales + scale_at(p, src, h);
            uint8_t* d = p.c.scales + scale_at(p, dst, h);
            d[0] = s[0];
            d[16] = s[16];
        }
    }
    const int n = __popc(__ballot_sync(0xFFFFFFFFu, from >= 0));  // (the first lanes)
    const long long side = (long long)p.c.page * ROWB;            // from a key to its value
    // where the lane's row begins
    const long long s0 = (((long long)src.page * p.c.Hkv + h) * 2 * p.c.page + src.slot) * ROWB;
    const long long d0 = (((long long)dst.page * p.c.Hkv + h) * 2 * p.c.page + dst.slot) * ROWB;
    const int sub = lane / kLanes, off = 16 * (lane % kLanes);
    for (int r = 0; r < 2 * n; r += kAhead * kAtOnce) {  // rows: the keys, then the values, of row r / 2
        uint4 v[kAhead];
        long long to[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int x = r + k * kAtOnce + sub, who = min(x / 2, 31);
            const long long s = __shfl_sync(0xFFFFFFFFu, s0, who) + (x % 2) * side + off;
            to[k] = __shfl_sync(0xFFFFFFFFu, d0, who) + (x % 2) * side + off;
            if (!__shfl_sync(0xFFFFFFFFu, (int)ok, who) || x >= 2 * n) to[k] = -1;
            else v[k] = *reinterpret_cast<const uint4*>(p.c.pages + s);
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (to[k] >= 0) *reinterpret_cast<uint4*>(p.c.pages + to[k]) = v[k];
    }
}

// In place: a block takes a head's keys (blockIdx.y 0) or values from front to back, kRows rows a round.  A round's loads
// are all done (the barrier) before its first store; the next round's may come before them too: rows are read at
// their place or behind it.
constexpr int kPlaceThreads = 512;
template <int ROWB>
__global__ void __launch_bounds__(kPlaceThreads) move_in_place_kernel(const __grid_constant__ EvictParams p) {
    constexpr int kLanes = ROWB / 16, kEach = 4, kStep = kPlaceThreads / kLanes, kRows = kEach * kStep;
    const int tid = threadIdx.x, unit = blockIdx.x, b = unit / p.c.Hkv, h = unit - b * p.c.Hkv, kv = blockIdx.y;
    wait_for_kernel_before();
    let_kernel_behind_in();
    const int stay = p.keep + p.recent;
    const int* row = p.t.pages + b * p.t.stride;
    const int* kept = p.kept + (long long)unit * stay;
    const int sub = tid / kLanes, off = 16 * (tid % kLanes);
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
            if (from == i) continue;
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
    const int grid = n_sm * (rt == 1 ? 2 : 1);
    auto go = [&](auto* f) { return launch_dependent(f, dim3((unsigned)grid), kThreads, 0, stream, p); };
    auto of_rows = [&](auto d, auto type) {
        constexpr int D = decltype(d)::value;
        constexpr bool E = decltype(type)::value;
        return rt == 1 ? go(weigh_kernel<D, E, 1>) : rt == 2 ? go(weigh_kernel<D, E, 2>) : go(weigh_kernel<D, E, 4>);
    };
    using D64 = std::integral_constant<int, 64>;
    using D128 = std::integral_constant<int, 128>;
    if (p.g.c.d == 64) return e4m3 ? of_rows(D64{}, std::true_type{}) : of_rows(D64{}, std::false_type{});
    return e4m3 ? of_rows(D128{}, std::true_type{}) : of_rows(D128{}, std::false_type{});
}

cudaError_t launch_evict(EvictParams p, bool e4m3, cudaStream_t stream) {
    const int units = p.B * p.c.Hkv, stay = p.keep + p.recent;
    p.cached = (int)std::min<long long>((long long)p.t.max_pages * p.c.page, kEvictCached);
    cudaError_t e = smem_opt_in(reinterpret_cast<const void*>(&rank_kernel), 4 * kEvictCached);
    if (e != cudaSuccess) return e;
    e = launch_dependent(rank_kernel, dim3((unsigned)units), kRankThreads, 4 * p.cached, stream, p);
    if (e != cudaSuccess) return e;
    const int rowb = p.c.d * (e4m3 ? 1 : 2);
    if (p.in_place) {
        const dim3 grid((unsigned)units, 2);
        auto go = [&](auto* f) { return launch_dependent(f, grid, kPlaceThreads, 0, stream, p); };
        return rowb == 64 ? go(move_in_place_kernel<64>) : rowb == 128 ? go(move_in_place_kernel<128>)
                                                                       : go(move_in_place_kernel<256>);
    }
    const int groups = (int)((std::min<long long>(stay, (long long)p.t.max_pages * p.c.page) + 31) / 32);
    const dim3 grid((unsigned)(((long long)units * groups + kWarps - 1) / kWarps));
    auto go = [&](auto* f) { return launch_dependent(f, grid, kThreads, 0, stream, p, groups); };
    return rowb == 64 ? go(move_kernel<64>) : rowb == 128 ? go(move_kernel<128>) : go(move_kernel<256>);
}

}  // namespace attn
