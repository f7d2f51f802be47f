// Decode attention for a batch whose sequences share long prefixes, each prefix's keys and values read once for all of its
// sequences.
//
//     O_i = sum_j softmax_j(scale q_i . k_j) v_j   over the prefix of row i's sequence, then the positions of its own.
//
// Three kernels.  The first attends to the prefixes: the rows of all members of a prefix, for one kv head, are the rows of
// a matrix, and a tile of 128 of them meets tiles of 128 positions,
//     S [128 x 128] = Q K^T,   O [128 x d] += P V,   P = 2^(scale' S - m),
// with tcgen05.mma: S and O in tensor memory, P written over S in 16 bits (weights of at most 2^8 relative to a reference m
// that moves only when a score passes it by 2^8; their sum is taken in float32 before they are rounded to bf16).  Over bf16 pages
// a weight is one bf16 number, off by 2^-8 of itself, where the decode kernel has two of them up to 32 rows to a head: O is 0.0023
// of its norm off the exact one instead of its own rounding's 0.0017.  Two would make three products of two (one with each half),
// 3900 clocks at the measured peak for two tiles of 128 x 128 that take 3800 now.  The decode
// kernels (attn_paged.cu, attn_paged_e4m3.cu) attend to the own positions and leave unscaled sums in float32.  The
// third joins the parts of every row: O = sum_k 2^(m_k - M) O_k / L, M = max m_k, L = sum_k 2^(m_k - M) l_k.
//
// Bound by the products and the exponentials where a prefix has many rows, by memory below about 150 rows: 4 flops a
// row and element read, against about 280 flops a byte.  Work is cut over one CTA a multiprocessor as in the decode
// kernels: units (prefix, kv head, up to 256 of the rows) end to end on a line of cost, equal shares of it.
//
// A CTA has two streams of scores -> weights -> output, so that one's products run under the other's exponentials.  With
// more than 128 rows the streams are two tiles of rows against the same positions (each tile of keys and values is
// loaded once for 256 rows), with up to 128 they are the same rows against the even and the odd tiles of positions, two
// parts to be joined.
//
//   warps 0-3, 4-7: a stream each, one thread a row: the queries to shared memory, weights, the row's part to global memory
//   bf16 pages: a warp for the TMA loads, boxes of 16 to 128 positions with 128 bytes of each row
//   E4M3 pages: a warp loads codes and exponents to places of their own, and four warps widen them to tiles of fp16 numbers,
//   relative to the tile's largest exponent (below).  Every operand is fp16 then: the queries relative to their row's
//   largest element, the weights relative to the largest product of weight and factor.  A pair of codes costs a
//   conversion and a product; as bf16 numbers, which need no common exponents, it was six instructions of warps that the
//   products wait for: 429 us for 4096 rows to a head behind 16K positions, now 328 (bf16 pages: 264), and 54.5 for 256 rows,
//   now 51.5.  Two of the warps take the keys and two the values (all four in turn: 354 us; codes loaded to registers by
//   the four themselves, a tile ahead, came late, 68 us for 256 rows).
//   last two warps: a stream each, one thread issues its products (one thread for both left gaps between them: a wait
//   that is already over costs it 130 cycles, four of them to 1030 cycles of products)
#include <cuda_bf16.h>

#include <cstddef>

#include "device_once.h"
#include "paged_device.h"

namespace attn {

using namespace ptx;

namespace {

constexpr int kTile = 128;         // rows of a stream, and positions of a tile
constexpr int kRows = 2 * kTile;   // of a unit, at most
// Costs are counted in products of a tile of rows with a tile of positions: w for a tile of positions, two or one, as there
// are rows; and what a unit costs beside them, `over`.
constexpr PagedShape kShape{kTile, 4, 4};

template <bool E4M3>
struct Roles {
    static constexpr int kWiden = 8, kLoad = E4M3 ? 12 : 8, kMma = kLoad + 1, kThreads = 32 * (kMma + 2);
};
struct Shared {
    unsigned cost[kPagedMaxBatch + 1];        // of the prefixes before g
    unsigned short members[kPagedMaxBatch + 1];  // sequences of the prefixes before g
    unsigned short order[kPagedMaxBatch];     // sequences by prefix
    unsigned short rank[kPagedMaxBatch];      // a sequence's place among those of its prefix
    short of[kPagedMaxBatch];                 // its prefix, -1: none
    unsigned count[kPagedMaxBatch];           // sequences of prefix g
    unsigned long long k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_half[2], p_full[2], o_full[2], q_full;
    unsigned long long c_full[3], c_empty[3];  // E4M3: places of codes
    alignas(16) uint8_t exps[3][kTile];
    int tile_exp[2][4];                       // E4M3: common exponents of tiles of keys and of values
    short q_exp[kRows];                       // and of the queries' rows
    unsigned scan[2][16];
    uint32_t tmem;
    int abort;
};
template <int D, bool E4M3>
struct Cfg {
    static constexpr int kKeyStages = E4M3 ? 1 : 2, kValueStages = 2, kCodeStages = 3;
    static constexpr int kParts = D / 64;           // of a row, 128 bytes each
    static constexpr int kPart = kTile * 128;
    static constexpr int kBytes = kParts * kPart;   // of a tile of queries, keys or values
    static constexpr int kCodes = kTile * D;        // of a tile of codes
    static constexpr int kOffK = 2 * kBytes, kOffV = kOffK + kKeyStages * kBytes, kOffCodes = kOffV + kValueStages * kBytes;
    static constexpr int kOffShared = kOffCodes + (E4M3 ? kCodeStages * kCodes : 0);
    static constexpr int kSmem = 1024 + kOffShared + (int)sizeof(Shared);
    static constexpr uint32_t kCols = 512, kColO = 256;  // scores of the streams at 0 and 128, outputs at 256 and 384
    static_assert(kSmem <= 232448, "shared memory");
};
constexpr float kRescale = 8.f;  // log2 of how far a score may pass the reference
// E4M3: tiles of codes become fp16 numbers, code * 2^(e - E + 7) with E the largest exponent of the tile's rows: 448 * 2^7 is the
// most, and factors of at least 2^-15 are exact.  Below that a code is rounded to a step of 2^-24, off by 2^-32 of 2^E at
// most: once, by a factor of 2^-24 or more as an fp16 number, by two (the first of them exact) for smaller ones.  Rows of the
// queries become fp16 numbers below 2^15.
constexpr int kUp = 7, kOne = 127 + kUp, kExact = -15, kSmallest = -24, kNothing = -34;  // (448 * 2^-34 is rounded to zero)
// Weights are fp16 numbers too, relative to a reference M of weight times 2^E: from 2^7 for the largest when M moves, up to 2^15.
constexpr float kMost = 15.f, kFirst = 7.f;
// A tile of values has an exponent of at least the largest so far less kApart, so that the weights of a tile of tiny
// values stay numbers; what is lost is below 2^-72 of the largest factor.
constexpr int kApart = 40;

__device__ __forceinline__ void tma_load_box(uint32_t dst, const CUtensorMap* map, uint32_t bar, int slot, int part, int kv,
                                             int unit) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(slot), "r"(part), "r"(kv), "r"(unit), "r"(bar)
        : "memory");
}

__device__ __forceinline__ int followed(const PrefixParams& p, int n) { return n < 0 || n > p.t.max_pages * p.c.page ? 0 : n; }
__device__ __forceinline__ int prefix_length(const PrefixParams& p, int g) { return followed(p, p.t.len[g]); }
__device__ __forceinline__ int prefix_of(const PrefixParams& p, int b) {
    const int g = p.of[b];
    return g < 0 || g >= p.G ? -1 : g;
}
__device__ __forceinline__ int tiles_of(int n) { return (n + kTile - 1) / kTile; }
// Units of one prefix and kv head: `whole` of 256 rows, and one of the rest (up to 128 rows cost half).
struct HeadCost {
    int whole, rest;     // units of 256 rows; rows of the last one, 0: none
    unsigned per, last;  // their costs
    __device__ __forceinline__ HeadCost(int rows, int tiles, unsigned over) {
        const PagedShape shape{kTile, over, kShape.least};
        whole = rows / kRows;
        rest = rows - whole * kRows;
        per = paged_cost(2 * tiles, shape);
        last = rest == 0 ? 0 : rest > kTile ? per : paged_cost(tiles, shape);
    }
    __device__ __forceinline__ unsigned sum() const { return whole * per + last; }
};
// The line of cost and its cuts.
struct Line {
    unsigned W, C, over;
    __device__ __forceinline__ PagedCuts cuts() const {
        PagedCuts c(0, 0, 1, kShape);
        c.C = C;
        c.q = W / C;
        c.r = W - c.q * C;
        return c;
    }
};

// Members by prefix and costs, by all threads; CTA 0 leaves them for the joining kernel.
template <int THREADS>
__device__ __forceinline__ Line prefix_plan(const PrefixParams& p, Shared& sh) {
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    if (!p.of) {  // one prefix, of all sequences
        const int len = prefix_length(p, 0), n = tiles_of(len);
        Line line{0, 1, kShape.overhead};
        HeadCost head(p.B * p.rows, n, line.over);
        const unsigned units = p.Hkv * (head.whole + (head.rest > 0));
        const unsigned work = head.whole || head.rest > kTile ? 2 * n : n;  // of a unit
        const unsigned k = max(1u, min(gridDim.x / units, work / 2));
        if (n && (head.whole == 0 || head.rest == 0 || head.rest > kTile) && units <= gridDim.x &&
            (k < gridDim.x / units || 10 * units * k >= 9 * gridDim.x)) {
            // units of the same cost: k CTAs to each, and `over` such that the cuts fall on the units' ends (a CTA with two
            // stretches would fill its pipeline twice: 78 us for a 32K prefix, and 72.5 so), unless that leaves CTAs idle.  Only
            // here: with prefix_of the members and costs of prefixes are known after the scan below, and units of different
            // costs have no such cuts; a caller with one prefix for all leaves prefix_of out
            const unsigned share = (max(work, kShape.least) + 1 + k - 1) / k;
            line.over = share * k - max(work, kShape.least);
            head = HeadCost(p.B * p.rows, n, line.over);
            line.C = units * k;
        } else if (n) {
            line.C = PagedCuts(p.Hkv * head.sum(), units, gridDim.x, kShape).C;
        }
        line.W = p.Hkv * head.sum();
        for (int b = tid; b < p.B; b += THREADS) {
            sh.order[b] = (unsigned short)b;
            if (blockIdx.x == 0) p.place[b] = make_int2(0, b);
        }
        if (tid == 0) {
            sh.cost[0] = 0;
            sh.cost[1] = line.W;
            sh.members[0] = 0;
            sh.members[1] = (unsigned short)p.B;
            if (blockIdx.x == 0) {
                if (p.t.len[0] != len) atomicOr(p.c.err, kCacheErrPosition);
                p.groups[0] = make_int4(0, 0, p.B, n);
                p.groups[1] = make_int4((int)line.W, (int)line.C, (int)line.over, 0);
            }
        }
        __syncthreads();
        return line;
    }
    for (int g = tid; g < p.G; g += THREADS) sh.count[g] = 0;
    const int first_len = tid < p.G ? p.t.len[tid] : 0;  // (on its way meanwhile)
    for (int b = tid; b < p.B; b += THREADS) {
        const int g = prefix_of(p, b);
        sh.of[b] = (short)g;
        if (blockIdx.x == 0 && g < 0 && p.of[b] != -1) atomicOr(p.c.err, kCacheErrPosition);
    }
    __syncthreads();
    if (warp == 0) {
        for (int b0 = 0; b0 < p.B; b0 += 32) {
            const int b = b0 + lane;
            const int g = b < p.B ? sh.of[b] : -1;
            const unsigned same = __match_any_sync(0xFFFFFFFFu, g);
            if (g >= 0) {
                const unsigned before = sh.count[g];
                sh.rank[b] = (unsigned short)(before + __popc(same & ((1u << lane) - 1)));
                __syncwarp(same);
                if ((same >> lane) == 1u) sh.count[g] = before + __popc(same);  // the last of them
            }
            __syncwarp();
        }
    }
    __syncthreads();
    unsigned carry_c = 0, carry_m = 0;
    int own_units = 0;
    if (tid == 0) {
        sh.cost[0] = 0;
        sh.members[0] = 0;
    }
    for (int g0 = 0; g0 < p.G; g0 += THREADS) {
        const int g = g0 + tid;
        unsigned c = 0, m = 0;
        if (g < p.G) {
            const int given = g0 ? p.t.len[g] : first_len, len = followed(p, given), n = tiles_of(len);
            if (blockIdx.x == 0 && given != len) atomicOr(p.c.err, kCacheErrPosition);
            m = sh.count[g];
            const HeadCost head((int)m * p.rows, n, kShape.overhead);
            c = p.Hkv * head.sum();
            if (n) own_units += p.Hkv * (head.whole + (head.rest > 0));
        }
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const unsigned y = __shfl_up_sync(0xFFFFFFFFu, c, o), z = __shfl_up_sync(0xFFFFFFFFu, m, o);
            if (lane >= o) {
                c += y;
                m += z;
            }
        }
        if (lane == 31) {
            sh.scan[0][warp] = c;
            sh.scan[1][warp] = m;
        }
        __syncthreads();
        unsigned all_c = carry_c, all_m = carry_m;
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) {
            if (w < warp) {
                c += sh.scan[0][w];
                m += sh.scan[1][w];
            }
            all_c += sh.scan[0][w];
            all_m += sh.scan[1][w];
        }
        if (g < p.G) {
            sh.cost[g + 1] = carry_c + c;
            sh.members[g + 1] = (unsigned short)(carry_m + m);
        }
        carry_c = all_c;
        carry_m = all_m;
        __syncthreads();
    }
#pragma unroll
    for (int o = 16; o; o /= 2) own_units += __shfl_xor_sync(0xFFFFFFFFu, own_units, o);
    if (lane == 0) sh.scan[0][warp] = own_units;
    for (int b = tid; b < p.B; b += THREADS) {
        const int g = sh.of[b], r = sh.rank[b];
        if (g >= 0) sh.order[sh.members[g] + r] = (unsigned short)b;
        if (blockIdx.x == 0) p.place[b] = g < 0 ? make_int2(-1, 0) : make_int2(g, r);
    }
    __syncthreads();
    unsigned units = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) units += sh.scan[0][w];
    const Line line{carry_c, PagedCuts(carry_c, units, gridDim.x, kShape).C, kShape.overhead};
    if (blockIdx.x == 0) {
        for (int g = tid; g < p.G; g += THREADS)
            p.groups[g] = make_int4((int)sh.cost[g], sh.members[g], sh.members[g + 1] - sh.members[g],
                                    tiles_of(prefix_length(p, g)));
        if (tid == 0) p.groups[p.G] = make_int4((int)line.W, (int)line.C, (int)line.over, 0);
    }
    return line;
}

// A CTA's part of a unit: tiles [g0, g1) of prefix g for rows of kv head h, from row `row0` of the prefix's rows on.
struct Stretch {
    unsigned at, end;
    int g, h, row0, rows, len, g0, g1;
    __device__ __forceinline__ bool two() const { return rows > kTile; }  // tiles of rows; else the streams share the positions
    // Tiles of a stream, and its i-th.
    __device__ __forceinline__ int steps(int stream) const { return two() ? g1 - g0 : (g1 - g0 + 1 - stream) / 2; }
    __device__ __forceinline__ int tile(int stream, int i) const { return g0 + (two() ? i : 2 * i + stream); }
};
__device__ __forceinline__ Stretch stretch_begin(const PrefixParams& p, const PagedCuts& cuts, const Shared& sh) {
    Stretch s{};
    s.at = cuts.begin(blockIdx.x);
    s.end = cuts.begin(blockIdx.x + 1);
    int lo = 0, hi = p.G - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (sh.cost[mid] <= s.at) lo = mid;
        else hi = mid - 1;
    }
    s.g = lo;
    return s;
}
__device__ __forceinline__ void stretch_open(const PrefixParams& p, const Shared& sh, unsigned over, Stretch& s) {
    while (sh.cost[s.g + 1] <= s.at) ++s.g;
    s.len = prefix_length(p, s.g);
    const int n = tiles_of(s.len), all = (sh.members[s.g + 1] - sh.members[s.g]) * p.rows;
    const HeadCost head(all, n, over);
    const unsigned into = s.at - sh.cost[s.g], sum = head.sum();
    s.h = (int)(into / sum);
    const unsigned in_head = into - s.h * sum;
    const int unit = min(head.whole, (int)(in_head / head.per));
    const unsigned off = in_head - unit * head.per, per = unit < head.whole ? head.per : head.last;
    const unsigned to = min(per, off + (s.end - s.at));
    s.row0 = unit * kRows;
    s.rows = min(kRows, all - s.row0);
    const int w = s.two() ? 2 : 1;
    s.g0 = min(n, max(0, (int)off - (int)over) / w);
    s.g1 = min(n, max(0, (int)to - (int)over) / w);
    s.at += to - off;
}

// Scores of 32 columns; those from `live` on become -inf.
template <bool MASKED, int OFF, int N>
__device__ __forceinline__ void mask_columns(uint32_t (&r)[N], int c0, int live) {
    if (MASKED) {
#pragma unroll
        for (int e = 0; e < 32; ++e)
            if (c0 + e >= live) r[OFF + e] = 0xFF800000u;
    }
}
template <int OFF, int N>
__device__ __forceinline__ float max_columns(const uint32_t (&r)[N], float m) {
    float x[4] = {m, m, m, m};
#pragma unroll
    for (int e = 0; e < 32; e += 2) x[(e >> 1) & 3] = fmax3(x[(e >> 1) & 3], __uint_as_float(r[OFF + e]), __uint_as_float(r[OFF + e + 1]));
    return fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
}
// Largest of a row's scores.  The first KEEP columns stay in registers for the weights.  A load from tensor memory is under way
// while the columns before are looked at.
template <bool MASKED, int KEEP>
__device__ __forceinline__ float row_max(uint32_t t_s, int live, uint32_t (&kept)[KEEP]) {
    float m = __int_as_float(0xFF800000);
    uint32_t r[2][32];
    tmem_ld32(t_s + KEEP, r[0]);
    tmem_wait_ld();
#pragma unroll
    for (int c0 = KEEP; c0 < kTile; c0 += 32) {
        constexpr int kLast = kTile - 32;
        uint32_t(&now)[32] = r[(c0 - KEEP) / 32 % 2];
        if (c0 < kLast) {
            tmem_ld32(t_s + c0 + 32, r[((c0 - KEEP) / 32 + 1) % 2]);
        } else {
            tmem_ld32_at<0>(t_s, kept);
            if constexpr (KEEP == 64) tmem_ld32_at<KEEP - 32>(t_s + 32, kept);
        }
        mask_columns<MASKED, 0>(now, c0, live);
        m = max_columns<0>(now, m);
        tmem_wait_ld();
    }
    mask_columns<MASKED, 0>(kept, 0, live);
    m = max_columns<0>(kept, m);
    if constexpr (KEEP == 64) {
        mask_columns<MASKED, KEEP - 32>(kept, 32, live);
        m = max_columns<KEEP - 32>(kept, m);
    }
    return m;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t y;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
    return y;
}
// Weights 2^(s scale - ref) of 32 columns as pairs of 16-bit numbers; their sum is added to `sum`.
template <bool F16, int OFF, int N>
__device__ __forceinline__ void weights32(const uint32_t (&r)[N], float2 scale, float2 nref, float2 (&sum)[2], uint32_t (&pk)[16]) {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        const float2 x = __ffma2_rn(make_float2(__uint_as_float(r[OFF + 2 * e]), __uint_as_float(r[OFF + 2 * e + 1])), scale, nref);
        const float2 y = make_float2(ex2(x.x), ex2(x.y));
        sum[e % 2] = __fadd2_rn(sum[e % 2], y);
        pk[e] = F16 ? pack_f16x2(y.x, y.y) : pack_bf16x2(y.x, y.y);
    }
}
// A row's sums so far times `fix`.
template <int D>
__device__ __forceinline__ void scale_row(uint32_t t_o, float fix) {
#pragma unroll
    for (int c0 = 0; c0 < D; c0 += 32) {
        uint32_t r[32];
        tmem_ld32(t_o + c0, r);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * fix);
        tmem_st32(t_o + c0, r);
    }
    tmem_wait_st();
}
// A row's weights over its scores (P over columns that this thread has read); returns their sum.  The first half (64
// positions) is announced as soon as it is written.
template <bool MASKED, bool F16, int KEEP>
__device__ __forceinline__ float row_weights(uint32_t t_s, int live, float scale, float ref, uint32_t bar_half,
                                             const uint32_t (&kept)[KEEP]) {
    const float2 scale2 = make_float2(scale, scale), nref = make_float2(-ref, -ref);
    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    uint32_t r[2][32], pk[16];
    tmem_ld32(t_s + KEEP, r[0]);
    weights32<F16, 0>(kept, scale2, nref, sum, pk);
    tmem_wait_ld();
    tmem_st16(t_s, pk);
    if constexpr (KEEP == 64) {
        weights32<F16, KEEP - 32>(kept, scale2, nref, sum, pk);
        tmem_st16(t_s + 16, pk);
    }
#pragma unroll
    for (int c0 = KEEP; c0 < kTile; c0 += 32) {
        if (c0 == 64) {
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(bar_half);
        }
        uint32_t(&now)[32] = r[(c0 - KEEP) / 32 % 2];
        if (c0 + 32 < kTile) tmem_ld32(t_s + c0 + 32, r[((c0 - KEEP) / 32 + 1) % 2]);
        mask_columns<MASKED, 0>(now, c0, live);
        weights32<F16, 0>(now, scale2, nref, sum, pk);
        if (c0 + 32 < kTile) tmem_wait_ld();
        tmem_st16(t_s + c0 / 2, pk);
    }
    return (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
}

__device__ __forceinline__ uint4 lds16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void sts16(uint32_t addr, const uint4& v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// Eight fp16 numbers times f (two of them).
__device__ __forceinline__ void scale8(uint4& v, uint32_t f) {
    asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(v.x) : "r"(f));
    asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(v.y) : "r"(f));
    asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(v.z) : "r"(f));
    asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(v.w) : "r"(f));
}
// 16 codes as fp16 numbers times f (two of them), two 16-byte pieces.
__device__ __forceinline__ void widen16(const uint4& v, uint32_t f, uint4& lo, uint4& hi) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(o[i]) : "h"((uint16_t)(w[i / 2] >> 16 * (i % 2))));
        asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(o[i]) : "r"(f));
    }
    lo = make_uint4(o[0], o[1], o[2], o[3]);
    hi = make_uint4(o[4], o[5], o[6], o[7]);
}
// The largest of a tile's exponents in front of position `live`; 255, a row of NaN, does not count.  By a whole warp.
__device__ __forceinline__ int largest_exponent(const uint8_t* exps, int live) {
    const int lane = threadIdx.x % 32;
    uint32_t four = *reinterpret_cast<const uint32_t*>(exps + 4 * lane);
    four = ((four & 0x7F7F7F7Fu) + 0x01010101u) ^ (four & 0x80808080u);  // one more, 0 for 255
    if (live < 4 * lane + 4) four &= live <= 4 * lane ? 0u : 0xFFFFFFFFu >> (32 - 8 * (live - 4 * lane));
    const uint32_t most = max(max(four & 255u, four >> 8 & 255u), max(four >> 16 & 255u, four >> 24));
    return max(0, (int)__reduce_max_sync(0xFFFFFFFFu, most) - 1);
}
// 2^x, x <= kUp, as two fp16 numbers; below 2^-24 zero.
__device__ __forceinline__ uint32_t half_power(int x) {
    return (x >= -14 ? (uint32_t)(x + 15) << 10 : x >= -24 ? 1u << (x + 24) : 0u) * 0x10001u;
}
// The bits of the largest finite magnitude of 8 bf16 numbers.
__device__ __forceinline__ uint32_t largest_bits(const uint4& v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = w[i] & 0x7FFFu, hi = w[i] >> 16 & 0x7FFFu;
        most = max(most, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
    }
    return most;
}
// 8 bf16 numbers times f as fp16 numbers.
__device__ __forceinline__ uint4 to_f16(const uint4& v, float f) {
    auto two = [&](uint32_t w) { return pack_f16x2(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xFFFF0000u) * f); };
    return make_uint4(two(v.x), two(v.y), two(v.z), two(v.w));
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(Roles<E4M3>::kThreads, 1) prefix_kernel(const __grid_constant__ PrefixParams p) {
    using C = Cfg<D, E4M3>;
    using R = Roles<E4M3>;
    constexpr int kKeyStages = C::kKeyStages, kValueStages = C::kValueStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* const smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    Shared& sh = *reinterpret_cast<Shared*>(smem + C::kOffShared);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const uint32_t s_q = smem_u32(smem), s_k = s_q + C::kOffK, s_v = s_q + C::kOffV;
    if (tid == 0) {
        prefetch_tmap(&p.tm);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sh.k_full[i]), E4M3 ? 2 : 1);
            mbar_init(smem_u32(&sh.v_full[i]), E4M3 ? 2 : 1);
            mbar_init(smem_u32(&sh.k_empty[i]), 2);
            mbar_init(smem_u32(&sh.v_empty[i]), 2);
        }
        for (int i = 0; i < C::kCodeStages; ++i) {
            mbar_init(smem_u32(&sh.c_full[i]), 1);
            mbar_init(smem_u32(&sh.c_empty[i]), 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sh.s_full[i]), 1);
            mbar_init(smem_u32(&sh.p_half[i]), 128);
            mbar_init(smem_u32(&sh.p_full[i]), 128);
            mbar_init(smem_u32(&sh.o_full[i]), 1);
        }
        mbar_init(smem_u32(&sh.q_full), 8);
        sh.abort = 0;
    }
    fence_barrier_init();
    wait_for_kernel_before();
    const Line line = prefix_plan<R::kThreads>(p, sh);
    const PagedCuts cuts = line.cuts();
    const unsigned over = line.over;
    let_kernel_behind_in();
    if (blockIdx.x >= cuts.C || line.W == 0) return;
    if (warp == R::kMma) {
        tmem_alloc(smem_u32(&sh.tmem), C::kCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&sh.tmem);
    const Watch watch{&sh.abort, p.c.err, p.watchdog_ns};
    Stretch s = stretch_begin(p, cuts, sh);

    if (warp < 8) {
        // =================================================== rows
        const int stream = warp / 4, row = tid % 128;
        const uint32_t t_lane = tmem + ((uint32_t)(warp % 4 * 32) << 16);
        const uint32_t t_s = t_lane + stream * kTile, t_o = t_lane + C::kColO + stream * kTile;
        const uint32_t s_full = smem_u32(&sh.s_full[stream]), p_half = smem_u32(&sh.p_half[stream]);
        const uint32_t p_full = smem_u32(&sh.p_full[stream]), o_full = smem_u32(&sh.o_full[stream]);
        const float ninf = __int_as_float(0xFF800000);
        constexpr int kKeep = E4M3 ? 32 : 64;  // (as the registers allow)
        int n = 0, stretch = 0, tiles = 0;  // the stream's tiles and stretches, all tiles of the stretches before
        while (s.at < s.end) {
            stretch_open(p, sh, over, s);
            if (s.g0 >= s.g1) continue;
            // ---- the queries, 16-byte pieces of rows in the layout of the products (128-byte swizzle), once both streams
            // are through with those before
            named_bar_sync(1, 256);
            constexpr int kLanes = D / 8, kAtOnce = 256 / kLanes, kBatch = kTile / kAtOnce;  // rows at once; a stream's rounds
            const int members0 = sh.members[s.g];
            for (int r0 = tid / kLanes; r0 < (s.two() ? 2 : 1) * kTile; r0 += kTile) {
                const int c = tid % kLanes;
                uint4 v[kBatch];
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    const int r = r0 + k * kAtOnce;
                    v[k] = make_uint4(0, 0, 0, 0);
                    if (r >= s.rows) continue;
                    const int x = s.row0 + r, member = x / p.rows;
                    const long long b = sh.order[members0 + member];
                    v[k] = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p.q) +
                                                           ((b * p.Hkv + s.h) * p.rows + (x - member * p.rows)) * D + 8 * c);
                }
                if (E4M3) {
                    uint32_t most[kBatch];
#pragma unroll
                    for (int k = 0; k < kBatch; ++k) most[k] = largest_bits(v[k]);
#pragma unroll
                    for (int x = kLanes / 2; x > 0; x /= 2)
#pragma unroll
                        for (int k = 0; k < kBatch; ++k) most[k] = max(most[k], __shfl_xor_sync(0xFFFFFFFFu, most[k], x));
#pragma unroll
                    for (int k = 0; k < kBatch; ++k) {
                        const int up = min(141 - (int)(most[k] >> 7), 127);  // the row's numbers come below 2^15
                        v[k] = to_f16(v[k], __uint_as_float((uint32_t)(up + 127) << 23));
                        if (c == 0) sh.q_exp[r0 + k * kAtOnce] = (short)-up;
                    }
                }
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    const int r = r0 + k * kAtOnce;
                    *reinterpret_cast<uint4*>(smem + (r / kTile) * C::kBytes + (c / 8) * C::kPart + (r % kTile) * 128 +
                                              ((c % 8) ^ (r & 7)) * 16) = v[k];
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.q_full));
            int q_exp = 0;
            if (E4M3) {
                named_bar_sync(1, 256);
                q_exp = sh.q_exp[s.two() ? stream * kTile + row : row];
            }
            const int steps = s.steps(stream);
            float m = ninf, l = 0.f, M = ninf;  // (M: E4M3)
            for (int i = 0; i < steps; ++i, ++n) {
                const int live = s.len - s.tile(stream, i) * kTile, t = tiles + s.tile(stream, i) - s.g0;
                wait(s_full, n & 1, watch);
                __syncwarp();
                tc_fence_after();
                uint32_t kept[kKeep];
                float scale = p.scale_log2;
                if (E4M3) {  // in the units of the row and the tile, a positive number whatever these are
                    const int x = q_exp + *reinterpret_cast<volatile int*>(&sh.tile_exp[0][t % 4]) - kOne;
                    scale = fminf(fmaxf(scale * __uint_as_float((uint32_t)(max(-126, min(x, 96)) + 127) << 23), 1.2e-38f), 3e38f);
                }
                const float top =
                    (live >= kTile ? row_max<false>(t_s, live, kept) : row_max<true>(t_s, live, kept)) * scale;
                if constexpr (E4M3) {
                    wait(smem_u32(&sh.v_full[t % kValueStages]), (t / kValueStages) & 1, watch);
                    __syncwarp();
                    const float ev = (float)*reinterpret_cast<volatile int*>(&sh.tile_exp[1][t % 4]);
                    // the reference of weight times factor moves (as below; a whole number, so that M - ev is exact)
                    if (__any_sync(0xFFFFFFFFu, top + ev > M + kMost)) {
                        const float to = fmaxf(M, ceilf(top + ev) - kFirst);
                        const float fix = to == M ? 1.f : ex2(M - to);
                        M = to;
                        if (i > 0) scale_row<D>(t_o, fix);
                    }
                    const float ref = M == ninf ? 0.f : M - ev;
                    const float sum = live >= kTile ? row_weights<false, true>(t_s, live, scale, ref, p_half, kept)
                                                    : row_weights<true, true>(t_s, live, scale, ref, p_half, kept);
                    tmem_wait_st();
                    tc_fence_before();
                    mbar_arrive(p_full);
                    // the sum of the weights, relative to the largest score
                    const float to = fmaxf(m, top);
                    if (to != ninf) l = (m == to ? l : l * ex2(m - to)) + sum * ex2(ref - to);
                    m = to;
                    continue;
                }
                // the reference moves, for all rows of the warp together, when a score passes it by 2^8 (the values of the
                // tile before are added by now: these scores were issued behind them)
                if (__any_sync(0xFFFFFFFFu, top > m + kRescale)) {
                    const float to = fmaxf(m, top);
                    const float fix = to == m ? 1.f : ex2(m - to);
                    m = to;
                    l *= fix;
                    if (i > 0) scale_row<D>(t_o, fix);
                }
                if (live < kTile) {
                    // positions past the end may hold anything: weight zero times a NaN is a NaN, so their values become
                    // zero (by either stream: neither waits for the other)
                    const int st = t % kValueStages;
                    wait(smem_u32(&sh.v_full[st]), (t / kValueStages) & 1, watch);
                    if (row >= live)
#pragma unroll
                        for (int x = 0; x < 8 * C::kParts; ++x)
                            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                             s_v + st * C::kBytes + (x / 8) * C::kPart + row * 128 + (x % 8) * 16),
                                         "r"(0)
                                         : "memory");
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                const float ref = m == ninf ? 0.f : m;
                l += live >= kTile ? row_weights<false, false>(t_s, live, scale, ref, p_half, kept)
                                   : row_weights<true, false>(t_s, live, scale, ref, p_half, kept);
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(p_full);
            }
            tiles += s.g1 - s.g0;
            // ---- the row's part: unscaled sums, reference and sum of weights
            const bool mine = s.two() ? stream * kTile + row < s.rows : row < s.rows;
            const int all = (sh.members[s.g + 1] - members0) * p.rows;
            const long long at = 2 * ((long long)p.Hkv * p.rows * members0 + (long long)s.h * all + s.row0) +
                                 stream * (s.two() ? kTile : s.rows) + row + (long long)kRows * blockIdx.x;
            if (mine) p.part_ml[at] = make_float2(m, l);
            wait(o_full, stretch++ & 1, watch);  // (without tiles, too: the thread of the products has been through the stretch)
            __syncwarp();
            tc_fence_after();
            if (steps == 0) continue;
            float* o = p.part_o + at * D;
            const float half = !E4M3 || m == ninf ? 1.f : ex2(0.5f * (M - m - kOne));  // (its square may pass a float's range)
#pragma unroll
            for (int c0 = 0; c0 < D; c0 += 32) {
                uint32_t r[32];
                tmem_ld32(t_o + c0, r);
                tmem_wait_ld();
                if (E4M3)
#pragma unroll
                    for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * half * half);
                if (mine) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8)
                        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(o + c0 + e), "r"(r[e]),
                                     "r"(r[e + 1]), "r"(r[e + 2]), "r"(r[e + 3]), "r"(r[e + 4]), "r"(r[e + 5]), "r"(r[e + 6]),
                                     "r"(r[e + 7])
                                     : "memory");
                }
            }
            tc_fence_before();
        }
    } else if (!E4M3 && warp == R::kLoad) {
        // =================================================== loads, a box or more to a lane
        const int box = p.box_rows, copies = kTile / box * C::kParts;  // of a tile of keys, at most 16
        const int mine = lane / C::kParts * box, part = lane % C::kParts;
        int n = 0;
        bool ok = true;
        while (s.at < s.end && ok) {
            stretch_open(p, sh, over, s);
            auto page_at = [&](int g) {
                const int pos = g * kTile + mine;
                if (lane >= copies || g >= s.g1 || pos >= s.len) return -1;
                int page = p.t.pages[s.g * p.t.stride + (unsigned)pos / (unsigned)p.c.page];
                if (page < 0 || page >= p.c.n_pages) {
                    atomicOr(p.c.err, kCacheErrPage);
                    page = 0;
                }
                return page;
            };
            int page = page_at(s.g0);
            for (int g = s.g0; g < s.g1 && ok; ++g, ++n) {
                const int next = page_at(g + 1);
                const bool need = page >= 0;
                const int slot = (int)((unsigned)(g * kTile + mine) % (unsigned)p.c.page), unit = page * p.Hkv + s.h;
                const int bytes = __popc(__ballot_sync(0xFFFFFFFFu, need)) * box * 128;
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    const int stages = kv ? kValueStages : kKeyStages, st = n % stages;
                    const uint32_t full = smem_u32(kv ? &sh.v_full[st] : &sh.k_full[st]);
                    if (ok && n >= stages)
                        ok = wait(smem_u32(kv ? &sh.v_empty[st] : &sh.k_empty[st]), (n / stages - 1) & 1, watch);
                    if (n + 1 == p.withhold) ok = false;
                    if (!__all_sync(0xFFFFFFFFu, ok)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) mbar_arrive_expect_tx(full, bytes);
                    __syncwarp();
                    if (need)
                        tma_load_box((kv ? s_v : s_k) + st * C::kBytes + part * C::kPart + mine * 128, &p.tm, full, slot, part,
                                     kv, unit);
                }
                page = next;
            }
        }
    } else if (warp == R::kLoad) {
        // =================================================== E4M3: codes and exponents, 16 positions to each of eight lanes
        const int box = p.box_rows, row = 16 * lane;
        const uint32_t codes0 = smem_u32(smem) + C::kOffCodes;
        int n = 0;  // tiles of keys and of values
        bool ok = true;
        while (s.at < s.end && ok) {
            stretch_open(p, sh, over, s);
            auto page_at = [&](int g) {
                const int pos = g * kTile + row;
                if (lane >= 8 || g >= s.g1 || pos >= s.len) return -1;
                int page = p.t.pages[s.g * p.t.stride + (unsigned)pos / (unsigned)p.c.page];
                if (page < 0 || page >= p.c.n_pages) {
                    atomicOr(p.c.err, kCacheErrPage);
                    page = 0;
                }
                return page;
            };
            int page = page_at(s.g0);
            for (int g = s.g0; g < s.g1 && ok; ++g) {
                const int next = page_at(g + 1);
                const int slot = (int)((unsigned)(g * kTile + row) % (unsigned)p.c.page), unit = page * p.Hkv + s.h;
                const bool need = page >= 0, head = need && row % box == 0;  // a box begins here
                const int bytes = __popc(__ballot_sync(0xFFFFFFFFu, head)) * box * D + __popc(__ballot_sync(0xFFFFFFFFu, need)) * 16;
#pragma unroll
                for (int kv = 0; kv < 2; ++kv, ++n) {
                    const int st = n % C::kCodeStages;
                    const uint32_t full = smem_u32(&sh.c_full[st]);
                    if (ok && n >= C::kCodeStages) ok = wait(smem_u32(&sh.c_empty[st]), (n / C::kCodeStages - 1) & 1, watch);
                    if (n / 2 + 1 == p.withhold) ok = false;
                    if (!__all_sync(0xFFFFFFFFu, ok)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) mbar_arrive_expect_tx(full, bytes);
                    __syncwarp();
                    if (head)
                        asm volatile(
                            "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                            " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(codes0 + st * C::kCodes + row * D),
                            "l"(reinterpret_cast<uint64_t>(&p.tm)), "r"(0), "r"(slot), "r"(kv), "r"(unit), "r"(full)
                            : "memory");
                    if (need)
                        asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], 16, [%2];" ::"r"(
                                         smem_u32(&sh.exps[st][row])),
                                     "l"(p.c.scales + ((long long)unit * (p.c.page / 16) + slot / 16) * 32 + 16 * kv), "r"(full)
                                     : "memory");
                }
                page = next;
            }
        }
    } else if (warp < R::kLoad) {
        // =================================================== E4M3: codes to tiles of fp16 numbers, two warps the keys', two the
        // values': a tile's waits, loads and fence are a chain of 1000 clocks and more, and so two of them run at once
        constexpr int kLanes = D / 16, kAtOnce = 64 / kLanes, kEach = kTile / kAtOnce;  // lanes of a row, rows at once
        static_assert(kEach == 2 * kLanes, "a lane has the factors of two rows");
        const int gtid = tid % 64, r0 = gtid / kLanes, c = gtid % kLanes, kv = warp / 2 % 2;
        const int stages = kv ? kValueStages : kKeyStages;
        const uint32_t codes0 = smem_u32(smem) + C::kOffCodes, places = kv ? s_v : s_k;
        const uint32_t full = smem_u32(kv ? sh.v_full : sh.k_full), empty = smem_u32(kv ? sh.v_empty : sh.k_empty);
        int n = kv, t = 0;  // tiles of keys and of values; of positions
        bool ok = true;
        while (s.at < s.end && ok) {
            stretch_open(p, sh, over, s);
            int most = 0;  // the largest exponent of the stretch's tiles of values
            for (int g = s.g0; g < s.g1; ++g, ++t, n += 2) {
                const int live = s.len - g * kTile, from = n % C::kCodeStages, st = t % stages;
                ok = wait(smem_u32(&sh.c_full[from]), (n / C::kCodeStages) & 1, watch);
                uint4 v[kEach];
#pragma unroll
                for (int i = 0; i < kEach; ++i) {
                    const int row = i * kAtOnce + r0, sw = D == 128 ? c ^ (row & 7) : c ^ ((row >> 1) & 3);
                    v[i] = make_uint4(0, 0, 0, 0);
                    if (row < live) v[i] = lds16(codes0 + from * C::kCodes + row * D + 16 * sw);
                }
                int top = largest_exponent(sh.exps[from], live);
                if (kv) {
                    most = max(most, top);
                    top = max(top, most - kApart);
                }
                uint32_t factor[2];  // of the lane's rows i = c and kLanes + c
                bool far = false;    // one of them is zero where two factors would not be
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int row = (x * kLanes + c) * kAtOnce + r0, e = sh.exps[from][row], power = e - top + kUp;
                    factor[x] = row >= live ? 0u : e == 255 ? 0x7E007E00u : half_power(power);  // (255: NaN)
                    far |= row < live && (unsigned)(power - kNothing - 1) < kSmallest - kNothing - 1;
                }
                if (ok && t >= stages) ok = wait(empty + 8 * st, (t / stages - 1) & 1, watch);
                const bool one = __all_sync(0xFFFFFFFFu, ok && !far);  // (one vote for both on the usual way)
                if (!one && !__all_sync(0xFFFFFFFFu, ok)) {
                    ok = false;
                    break;
                }
                __syncwarp();
                if (lane == 0 && one) mbar_arrive(smem_u32(&sh.c_empty[from]));  // (the warp's codes are in registers)
                // (of four tiles: keys come two tiles ahead of the weights, where a stream has every other tile)
                if (gtid == 0) *reinterpret_cast<volatile int*>(&sh.tile_exp[kv][t % 4]) = top;
                const uint32_t dst = places + st * C::kBytes + (c / 4) * C::kPart;
                auto store = [&](int row, const uint4& lo, const uint4& hi) {
                    // the lanes of a row's second half begin with the other piece: all 32 banks at once
                    const bool turned = c >= 4;
                    const int x = 2 * (c % 4);
                    const uint32_t at = dst + row * 128;
                    sts16(at + ((x + turned) ^ (row & 7)) * 16, turned ? hi : lo);
                    sts16(at + ((x + !turned) ^ (row & 7)) * 16, turned ? lo : hi);
                };
#pragma unroll
                for (int i = 0; i < kEach; ++i) {
                    uint4 lo, hi;
                    widen16(v[i], __shfl_sync(0xFFFFFFFFu, factor[i / kLanes], i % kLanes, kLanes), lo, hi);
                    store(i * kAtOnce + r0, lo, hi);
                }
                if (!one) {
                    // the rows that one factor takes to zero again, from the codes, in a loop of their own: a second factor in
                    // the usual one, or a second copy of that, took 342 to 375 us for 4096 rows behind 16K where nothing is
                    // far; 328 so (322 without any of this), and 416 where every tile has such rows
#pragma unroll 1
                    for (int i = 0; i < kEach; ++i) {
                        const int row = i * kAtOnce + r0, power = sh.exps[from][row] - top + kUp;
                        if (row >= live || power >= kSmallest || power <= kNothing) continue;
                        const int sw = D == 128 ? c ^ (row & 7) : c ^ ((row >> 1) & 3);
                        uint4 lo, hi;
                        widen16(lds16(codes0 + from * C::kCodes + row * D + 16 * sw), half_power(kExact), lo, hi);
                        scale8(lo, half_power(power - kExact));
                        scale8(hi, half_power(power - kExact));
                        store(row, lo, hi);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&sh.c_empty[from]));
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(full + 8 * st);
            }
        }
    } else {
        // =================================================== products of a stream (lane 0)
        if (lane == 0) {
            constexpr uint32_t idesc_s = E4M3 ? idesc_f16_f32(kTile, kTile, false) : idesc_bf16_f32(kTile, kTile, false);
            constexpr uint32_t idesc_o = E4M3 ? idesc_f16_f32(kTile, D, true) : idesc_bf16_f32(kTile, D, true);
            const int stream = warp - R::kMma;
            const uint32_t t_s = tmem + stream * kTile, t_o = tmem + C::kColO + stream * kTile;
            const uint32_t s_full = smem_u32(&sh.s_full[stream]), p_half = smem_u32(&sh.p_half[stream]);
            const uint32_t p_full = smem_u32(&sh.p_full[stream]), k_full = smem_u32(sh.k_full), v_full = smem_u32(sh.v_full);
            const uint32_t k_empty = smem_u32(sh.k_empty), v_empty = smem_u32(sh.v_empty);
            int n = 0, stretch = 0, done = 0;  // all tiles of the stretches before; the stream's
            bool ok = true;
            while (s.at < s.end && ok) {
                stretch_open(p, sh, over, s);
                if (s.g0 >= s.g1) continue;
                const bool two = s.two();
                const int steps = s.steps(stream);
                const uint32_t q = s_q + (two ? stream * C::kBytes : 0);
                ok = wait(smem_u32(&sh.q_full), stretch++ & 1, watch);
                // A stream without tiles announces its output all the same: the rows wait for it before they announce the next
                // stretch's queries, which would otherwise be the second phase of q_full since this thread last looked, and a
                // wait does not tell that from the first.
                if (ok && steps == 0) mbar_arrive(smem_u32(&sh.o_full[stream]));
                // Keys of a tile that the other stream uses, where there is one place for all: each stream sees every filling
                // of it (a wait tells one from the next, not from the one after that), and gives the place free.
                auto skip = [&](int t) {
                    if (t >= n + s.g1 - s.g0 || !(ok = ok && wait(k_full, t & 1, watch))) return;
                    mbar_arrive(k_empty);
                };
                // scores of tile t; their columns hold the weights of the tile before, whose product with the values, issued
                // earlier, has read them by the time they are written
                auto scores = [&](int t) {
                    const int st = t % kKeyStages;
                    if (!(ok = ok && wait(k_full + 8 * st, (t / kKeyStages) & 1, watch))) return;
                    tc_fence_after();
                    const uint32_t k0 = s_k + st * C::kBytes;
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t off = (k / 4) * C::kPart + (k % 4) * 32;
                        mma_ss(t_s, sdesc_sw128(q + off, 16, 1024), sdesc_sw128(k0 + off, 16, 1024), idesc_s, k > 0);
                    }
                    mma_commit(s_full);
                    mma_commit(k_empty + 8 * st);
                    if (two) return;
                    if (kKeyStages > 1) mma_commit(k_empty + 8 * st);  // for the other stream, which does not look at it
                    else skip(t + 1);
                };
                int t = two ? n : n + stream;
                if (!two && kKeyStages == 1 && stream == 1) skip(n);
                if (steps > 0) scores(t);
                for (int i = 0; i < steps && ok; ++i) {
                    const int st = t % kValueStages;
                    const uint32_t v = s_v + st * C::kBytes;
                    ok = wait(v_full + 8 * st, (t / kValueStages) & 1, watch) && wait(p_half, done & 1, watch);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_ts(t_o, t_s + 8 * k, sdesc_sw128(v + k * 16 * 128, C::kPart, 1024), idesc_o, i > 0 || k > 0);
                    if (!(ok = wait(p_full, done & 1, watch))) break;
                    tc_fence_after();
#pragma unroll
                    for (int k = 4; k < 8; ++k)
                        mma_ts(t_o, t_s + 8 * k, sdesc_sw128(v + k * 16 * 128, C::kPart, 1024), idesc_o, 1u);
                    ++done;
                    mma_commit(v_empty + 8 * st);
                    if (!two) mma_commit(v_empty + 8 * st);
                    t += two ? 1 : 2;
                    if (i + 1 < steps) scores(t);
                    else mma_commit(smem_u32(&sh.o_full[stream]));
                }
                n += s.g1 - s.g0;
            }
        }
        __syncwarp();
    }
    // all warps meet behind their last copy and product
    __syncthreads();
    if (sh.abort) {
        drain();
        __syncthreads();
    }
    if (warp == R::kMma) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kCols);
    }
}

// Joins a row's parts, a warp to a row: those of its prefix, from the CTAs that held tiles of its unit, and those of its
// own positions.
constexpr int kJoinWarps = 4;
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const __grid_constant__ PrefixParams p,
                                                               const __grid_constant__ JoinParams own) {
    constexpr int kVec = D / 32, kBatch = 8;
    wait_for_kernel_before();
    let_kernel_behind_in();
    const int lane = threadIdx.x % 32;
    const long long out = (long long)blockIdx.x * kJoinWarps + threadIdx.x / 32;  // row of O
    if (out >= (long long)p.B * p.Hkv * p.rows) return;
    const int head = (int)(out / p.rows), r = (int)(out - (long long)head * p.rows), b = head / p.Hkv, h = head - b * p.Hkv;
    const float ninf = __int_as_float(0xFF800000);
    // the prefix's parts
    int n1 = 0, c0 = 0, streams = 1, step = 0;
    long long base = 0;
    const int2 place = __ldcg(&p.place[b]);
    if (place.x >= 0) {
        const int4 g = __ldcg(&p.groups[place.x]), total = __ldcg(&p.groups[p.G]);
        const int all = g.z * p.rows, x = place.y * p.rows + r;
        if (g.w > 0) {
            const PagedCuts cuts = Line{(unsigned)total.x, (unsigned)total.y, 0}.cuts();
            const HeadCost head(all, g.w, total.z);
            const int unit = x / kRows, rows = min(kRows, all - unit * kRows), w = rows > kTile ? 2 : 1;
            const unsigned u0 = (unsigned)g.x + h * head.sum() + unit * head.per + total.z;
            // a tile is the CTA's that its last product's cost belongs to
            c0 = (int)cuts.owner(u0 + w - 1);
            streams = w == 2 ? 1 : 2;
            n1 = ((int)cuts.owner(u0 + w * g.w - 1) - c0 + 1) * streams;
            base = 2 * ((long long)p.Hkv * p.rows * g.y + (long long)h * all + unit * kRows) + x - unit * kRows;
            step = rows;
        }
    }
    // and its own
    const int row_block = r / own.rows_pad, unit = head * own.row_blocks + row_block;
    const int2 cut = __ldcg(&own.cut[unit]);
    const int n = n1 + (cut.x < 0 ? 1 : cut.y - cut.x + 1);
    auto find = [&](int i, const float*& o, float2& ml) {
        long long at;
        if (i < n1) {
            at = base + (long long)kRows * (c0 + i / streams) + i % streams * step;
            o = p.part_o + at * D;
            ml = __ldcg(&p.part_ml[at]);
        } else if (cut.x < 0) {
            o = own.whole_o + out * D;
            ml = __ldcg(&own.whole_ml[out]);
        } else {
            at = (long long)(2 * (cut.x + i - n1) + (i == n1)) * own.rows_pad + (r - row_block * own.rows_pad);
            o = own.part_o + at * D;
            ml = __ldcg(&own.part_ml[at]);
        }
    };
    float M = ninf, L = 0.f, v[kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j) v[j] = 0.f;
    for (int i0 = 0; i0 < n; i0 += 32) {
        const float* o = nullptr;
        float2 ml = make_float2(ninf, 0.f);
        if (i0 + lane < n) find(i0 + lane, o, ml);
        float top = ml.x;
#pragma unroll
        for (int k = 16; k; k /= 2) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, k));
        const float to = fmaxf(M, top);
        const float fix = M == to ? 1.f : ex2(M - to);
        M = to;
        L *= fix;
#pragma unroll
        for (int j = 0; j < kVec; ++j) v[j] *= fix;
        // a part without a reference has seen nothing (sum 0: its output is not looked at), or only NaN
        const float f = ml.x == ninf ? ml.y : ex2(ml.x - M);
        L += ml.x == ninf ? ml.y : ml.y * f;
        const int m = min(32, n - i0);
        for (int k0 = 0; k0 < m; k0 += kBatch) {
            float y[kBatch][kVec];
            float w[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int who = min(k0 + k, 31);
                const float* src = reinterpret_cast<const float*>(
                    __shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(o), who));
                w[k] = __shfl_sync(0xFFFFFFFFu, f, who);
                if (k0 + k >= m) w[k] = 0.f;
#pragma unroll
                for (int j = 0; j < kVec; ++j) y[k][j] = 0.f;
                if (w[k] != 0.f) {
                    if constexpr (D == 128) {
                        const float4 t = __ldcg(reinterpret_cast<const float4*>(src) + lane);
                        y[k][0] = t.x; y[k][1] = t.y; y[k][kVec - 2] = t.z; y[k][kVec - 1] = t.w;
                    } else {
                        const float2 t = __ldcg(reinterpret_cast<const float2*>(src) + lane);
                        y[k][0] = t.x; y[k][1] = t.y;
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
#pragma unroll
                for (int j = 0; j < kVec; ++j) v[j] = fmaf(w[k], y[k][j], v[j]);
        }
    }
#pragma unroll
    for (int k = 16; k; k /= 2) L += __shfl_xor_sync(0xFFFFFFFFu, L, k);
    const float inv = L == 0.f ? 0.f : 1.f / L;
    uint32_t* dst = reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(own.o) + out * D) + lane * (D / 64);
#pragma unroll
    for (int j = 0; j < D / 64; ++j) dst[j] = pack_bf16x2(v[2 * j] * inv, v[2 * j + 1] * inv);
    if (own.lse && lane == 0) own.lse[out] = (M + log2f(L)) * 0.6931471805599453f;
}

}  // namespace

cudaError_t launch_prefix(const PrefixParams& p, bool e4m3, int grid, cudaStream_t stream) {
    auto go = [&](auto* f, int threads, int smem) {
        const cudaError_t e = smem_opt_in(reinterpret_cast<const void*>(f), smem);
        return e != cudaSuccess ? e : launch_dependent(f, dim3((unsigned)grid), threads, smem, stream, p);
    };
    if (p.c.d == 64)
        return e4m3 ? go(prefix_kernel<64, true>, Roles<true>::kThreads, Cfg<64, true>::kSmem)
                    : go(prefix_kernel<64, false>, Roles<false>::kThreads, Cfg<64, false>::kSmem);
    return e4m3 ? go(prefix_kernel<128, true>, Roles<true>::kThreads, Cfg<128, true>::kSmem)
                : go(prefix_kernel<128, false>, Roles<false>::kThreads, Cfg<128, false>::kSmem);
}

cudaError_t launch_join(const PrefixParams& p, const JoinParams& own, cudaStream_t stream) {
    const long long rows = (long long)p.B * p.Hkv * p.rows;
    const dim3 grid((unsigned)((rows + kJoinWarps - 1) / kJoinWarps));
    return p.c.d == 64 ? launch_dependent(join_kernel<64>, grid, 32 * kJoinWarps, 0, stream, p, own)
                       : launch_dependent(join_kernel<128>, grid, 32 * kJoinWarps, 0, stream, p, own);
}

}  // namespace attn
