// Attention of a few new rows per sequence over a paged E4M3 cache.
//
//     O_i = sum_j softmax_j(scale q_i . k_j) v_j,   k_j = 2^a_j K_j,  v_j = 2^b_j V_j   (K_j, V_j: rows of E4M3 codes)
//
// Bound by memory: 2 (d + 1) bytes a position and kv head, read once.  The work is cut over the CTAs as in attn_paged.cu.
//
// The codes go into the tensor cores as they are.  Turning them into 16-bit numbers in registers takes 1260 instructions
// for 32 positions and was the limit (141 us for 456 MB, 48% of the measured copy rate; m16n8k32 products do the same
// inside, and measured 118 us).  Here the 128 positions of a tile fill the product's M dimension and the rows of the
// kv head its N dimension,
//
//     S^T [128 x N] = K [128 x d] Q^T [d x N],     D^T [d x N] = V^T [d x 128] P^T [128 x N],
//
// with tcgen05.mma, both operands in shared memory.  Q and P are 16-bit numbers at least, so each is the sum of two
// E4M3 numbers, x = hi + lo / 16, in columns of their own: N = 2 * rows.  The two sums meet in float32:
//   Q: a row is scaled by a power of two to at most 2^8; the two parts hold all eight bits of a bf16 number, down to
//      2^-22 of the row's largest.
//   P: weights times the value factors, scaled for each tile and row so that the largest weight and the largest factor
//      together give 2^8; the two parts are within 2^-8 of a weight (a bf16 number's rounding) and 2^-22 of that.
// Thread t of a group of four computing warps owns position t of a tile (tensor-memory lane t), where both row factors
// are its own, and element t of D^T, for the group's rows: all of them up to 8, half of them, in two groups that share
// nothing but the tiles, above.  D^T is added to the thread's float32 output after every tile, in terms of a reference
// that moves only when a score passes it by 2^16; l is summed by position and added over the threads at the end.
//
//   computing warps: Q parts, S^T -> P parts, output      then one warp for the TMA loads, and one thread for the products
//
// S^T is double-buffered: the product of tile n + 1 runs while the weights of tile n are formed, and that of V with
// the weights of tile n runs while tile n + 1 is prepared.  Two CTAs a multiprocessor up to 16 rows, one above.
#include <cuda_bf16.h>

#include <cstddef>

#include "device_once.h"
#include "paged_device.h"

namespace attn {

using namespace ptx;

namespace {

constexpr int kKeys = 128;
constexpr int kMostStages = 8;

template <int RP>
struct Shared {
    static constexpr int kGroups = RP / 8, kThreads = 128 * kGroups + 64;
    unsigned cost[kPagedMaxBatch + 4];
    unsigned long long full[kMostStages], empty[kMostStages], s_full[2], s_free[2], p_full, d_full, q_full;
    alignas(16) float top[2][4][RP];  // a tile's row maxima, by warp
    alignas(16) float factor[2][kGroups][4];  // and its largest value exponent, by group and warp
    alignas(16) float qs[RP];         // what a row's product is multiplied by, 2^up * scale * log2 e
    alignas(16) int last[RP];         // the positions a row sees
    alignas(16) int first[RP];
    float sum[4][RP];
    unsigned scan[kThreads / 32];
    uint32_t tmem;
    int abort;
};

template <int D, int RP>
struct Cfg {
    static constexpr int kN = 2 * RP;
    static constexpr int kCtas = RP <= 16 ? 2 : 1;
    static constexpr int kGroups = Shared<RP>::kGroups, kThreads = Shared<RP>::kThreads;
    static constexpr int kRows = 8;                         // of a thread
    static constexpr int kTile = kKeys * D;                 // bytes of a tile's keys, or values
    static constexpr int kStage = 2 * kTile;
    static constexpr int kScale = 2 * kKeys;                // its exponents
    static constexpr int kZero = D == 64 ? 32 * 64 : 0;     // rows 64 .. 127 of V^T, for the product's 128 rows
    static constexpr int kQ = kN * D, kP = kN * kKeys;
    static constexpr int kLimit = kCtas == 2 ? 115712 : 232448;
    static constexpr int kFit = (kLimit - 1024 - kZero - kQ - kP - (int)sizeof(Shared<RP>)) / (kStage + kScale);
    static constexpr int kStages = kFit < kMostStages ? kFit : kMostStages;
    static constexpr int kOffZero = kStages * kStage, kOffQ = kOffZero + kZero, kOffP = kOffQ + kQ;
    static constexpr int kOffScale = kOffP + kP, kOffShared = kOffScale + kStages * kScale;
    static constexpr int kSmem = 1024 + kOffShared + (int)sizeof(Shared<RP>);
    static constexpr uint32_t kCols = 3 * kN <= 64 ? 64 : 3 * kN <= 128 ? 128 : 3 * kN <= 256 ? 256 : 512;
    static constexpr uint32_t kSwizzle = D == 128 ? 2 : 4;  // rows of 128 or 64 bytes
    static_assert(kStages >= 3 && kSmem <= kLimit && kCols * kCtas <= 512, "shared and tensor memory");
    static_assert(kOffP % 128 == 0 && kOffQ % 1024 == 0 && kOffScale % 16 == 0 && kOffShared % 16 == 0, "alignment");
};

__device__ __forceinline__ void tma_load_rows(uint32_t dst, const CUtensorMap* map, uint32_t bar, int slot, int kv,
                                              int unit) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(slot), "r"(kv), "r"(unit), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ float exponent_factor(uint32_t e) {  // 2^(e - 127); e = 255 (NaN codes beside it): inf
    return __uint_as_float(max(e << 23, 0x00400000u));
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t addr) {
    uint32_t e;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(e) : "r"(addr) : "memory");
    return e;
}
// 32 lanes x 8 columns of 32 bit
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
// Two floats of magnitude at most 2^8 as two E4M3 numbers each, x = hi + lo / 16, by way of fp16 (2^-11 of a number; what
// follows is exact up to lo's own rounding).
__device__ __forceinline__ void split2_e4m3(float x0, float x1, uint32_t& hi, uint32_t& lo) {
    asm("{\n\t.reg .b32 y, h, t;\n\t.reg .b16 e, f;\n\t"
        "cvt.rn.f16x2.f32 y, %3, %2;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 e, y;\n\t"
        "cvt.rn.f16x2.e4m3x2 h, e;\n\t"
        "mul.rn.f16x2 y, y, %4;\n\t"
        "fma.rn.f16x2 t, h, %5, y;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 f, t;\n\t"
        "cvt.u32.u16 %0, e;\n\tcvt.u32.u16 %1, f;\n\t}"
        : "=r"(hi), "=r"(lo)
        : "f"(x0), "f"(x1), "r"(0x4C004C00u), "r"(0xCC00CC00u));  // 16 and -16, twice
}
__device__ __forceinline__ float warp_max(float x) {
    float y;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}

// Eight rows of the thread's tensor-memory lane: the hi columns, and the lo columns RP further on.
template <int RP>
__device__ __forceinline__ void load_parts(uint32_t addr, float (&hi)[8], float (&lo)[8]) {
    uint32_t a[8], b[8];
    tmem_ld8(addr, a);
    tmem_ld8(addr + RP, b);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        hi[i] = __uint_as_float(a[i]);
        lo[i] = __uint_as_float(b[i]);
    }
}

template <int D, int RP>
__global__ void __launch_bounds__(Shared<RP>::kThreads, (RP <= 16 ? 2 : 1))
    paged_e4m3_kernel(const __grid_constant__ PagedParams p) {
    using C = Cfg<D, RP>;
    constexpr PagedShape shape = paged_shape(D, true);
    static_assert(shape.keys == kKeys, "a tile is a key block");
    constexpr int N = C::kN, kStages = C::kStages, kThreads = C::kThreads, kLoader = 4 * C::kGroups;
    constexpr int kRows = C::kRows;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* const smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    Shared<RP>& sh = *reinterpret_cast<Shared<RP>*>(smem + C::kOffShared);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const uint32_t s_stage = smem_u32(smem), s_zero = s_stage + C::kOffZero, s_q = s_stage + C::kOffQ;
    const uint32_t s_p = s_stage + C::kOffP, s_scale = s_stage + C::kOffScale;
    auto full = [&](int st) { return smem_u32(&sh.full[st]); };
    auto empty = [&](int st) { return smem_u32(&sh.empty[st]); };

    if (tid == 0) {
        prefetch_tmap(&p.tm);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sh.s_full[i]), 1);
            mbar_init(smem_u32(&sh.s_free[i]), 4 * C::kGroups);
        }
        mbar_init(smem_u32(&sh.p_full), 4 * C::kGroups);
        mbar_init(smem_u32(&sh.d_full), 1);
        mbar_init(smem_u32(&sh.q_full), 4 * C::kGroups);
        sh.abort = 0;
    }
    if (D == 64)
        for (int i = tid; i < C::kZero / 16; i += kThreads)
            *reinterpret_cast<uint4*>(smem + C::kOffZero + 16 * i) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    fence_barrier_init();
    wait_for_kernel_before();
    int busy;
    const unsigned W = paged_prefix<kKeys, kThreads>(p, shape, sh.cost, sh.scan, busy) * p.units;
    const PagedCuts cuts(W, busy * p.units, gridDim.x, shape);
    let_kernel_behind_in();
    if (busy < p.B) paged_empty_rows<D, kThreads>(p, sh.cost);
    if (tid == 0 && !p.by_unit) p.cut[blockIdx.x] = make_int2(-1, 0);
    if (blockIdx.x >= cuts.C || W == 0) return;
    const Watch watch{&sh.abort, p.c.err, p.watchdog_ns};
    Walk w = paged_begin(p, cuts, sh.cost);

    // The tensor memory's address, once it is allocated: called once by the computing warps and the allocating one, which
    // nobody waits for before (the loads are on their way and the queries written by then).
    auto tmem_ready = [&]() {
        tc_fence_before();
        named_bar_sync(1 + C::kGroups, kThreads - 32);
        tc_fence_after();
        return *reinterpret_cast<volatile uint32_t*>(&sh.tmem);
    };
    if (warp == kLoader) {
        // =================================================== loads: a batch of four tiles, eight lanes each
        int g = 0, st = 0, n = 0;
        const int box = p.box_rows, part = lane % 8;
        const uint32_t box_bytes = 2 * box * D + 2 * box;
        struct Batch {
            int tiles, unit, slot;
        };
        auto fetch = [&](Batch& f) {
            f.tiles = 0;
            while (g >= w.g1) {
                if (w.at >= w.end) return;
                paged_open<kKeys>(p, shape, sh.cost, w);
                g = w.g0;
            }
            f.tiles = min(4, w.g1 - g);
            const int pos = (w.lo + g + lane / 8) * kKeys + 16 * part;
            f.unit = -1;
            if (lane / 8 < f.tiles && 16 * part % box == 0 && pos < w.len && pos + box > w.seen) {
                const int index = (unsigned)pos / (unsigned)p.c.page;
                f.slot = pos - index * p.c.page;
                int page = p.t.pages[w.b * p.t.stride + index];
                if (page < 0 || page >= p.c.n_pages) {
                    atomicOr(p.c.err, kCacheErrPage);
                    page = 0;
                }
                f.unit = page * p.Hkv + w.h / (p.units / p.Hkv);
            }
            g += 4;
        };
        Batch now, then;
        fetch(now);
        bool ok = true;
        while (now.tiles && ok) {
            for (int i = 0; i < now.tiles; ++i, ++n) {
                if (n >= kStages) ok = wait(empty(st), (n / kStages - 1) & 1, watch);
                if (n + 1 == p.withhold) ok = false;
                if (!__all_sync(0xFFFFFFFFu, ok)) {
                    ok = false;
                    break;
                }
                const bool mine = lane / 8 == i && now.unit >= 0;
                const int boxes = __popc(__ballot_sync(0xFFFFFFFFu, mine));
                if (lane == 0) mbar_arrive_expect_tx(full(st), boxes * box_bytes);
                __syncwarp();
                if (mine) {
                    const uint32_t dst = s_stage + st * C::kStage + 16 * part * D;
                    tma_load_rows(dst, &p.tm, full(st), now.slot, 0, now.unit);
                    tma_load_rows(dst + C::kTile, &p.tm, full(st), now.slot, 1, now.unit);
                    bulk_load(s_scale + st * C::kScale + 32 * part,
                              p.c.scales + ((long long)now.unit * (p.c.page / 16) + now.slot / 16) * 32, 2 * box, full(st));
                }
                st = st + 1 == kStages ? 0 : st + 1;
                if (i == min(1, now.tiles - 1)) fetch(then);  // its page numbers: two tiles are on their way by now
            }
            now = then;
        }
    } else if (warp == kLoader + 1) {
        // =================================================== products (lane 0)
        tmem_alloc(smem_u32(&sh.tmem), C::kCols);
        tmem_relinquish();
        const uint32_t tmem = tmem_ready(), t_d = tmem + 2 * N;
        if (lane == 0) {
            constexpr uint32_t idesc_s = idesc_e4m3_f32(kKeys, N, false);
            // V: elements of d contiguous; P: columns contiguous, 16 bytes to a position
            constexpr uint32_t idesc_d = idesc_e4m3_f32(kKeys, N, true) | (1u << 15);
            constexpr uint32_t sbo = 8 * D;
            int n = 0, stretch = 0;
            bool ok = true;
            auto values = [&](int m) {  // D^T of tile m
                if (!(ok = wait(smem_u32(&sh.p_full), m & 1, watch))) return;
                tc_fence_after();
                const int st = m % kStages;
#pragma unroll
                for (int kk = 0; kk < kKeys / 32; ++kk) {
                    const uint32_t a = s_stage + st * C::kStage + C::kTile + kk * 32 * D;
                    const uint32_t lbo = D == 64 ? s_zero - a : 16;
                    // P: 16 columns of 8 positions are 128 bytes; the next 8 positions follow, the next 16 columns
                    // come behind all positions
                    mma_ss_f8(t_d, sdesc_sw(a, lbo, sbo, C::kSwizzle), sdesc_plain(s_p + 32 * 16 * kk, 128, 16 * kKeys),
                              idesc_d, kk > 0);
                }
                mma_commit(smem_u32(&sh.d_full));
                mma_commit(empty(st));
            };
            while (w.at < w.end && ok) {
                paged_open<kKeys>(p, shape, sh.cost, w);
                for (int g = w.g0; g < w.g1 && ok; ++g, ++n) {
                    const int st = n % kStages;
                    // the queries of a new stretch are written once the last tile before it is done
                    if (g == w.g0) {
                        if (n > 0) values(n - 1);
                        if (ok) ok = wait(smem_u32(&sh.q_full), stretch++ & 1, watch);
                    }
                    if (ok) ok = wait(full(st), (n / kStages) & 1, watch);
                    if (ok && n >= 2) ok = wait(smem_u32(&sh.s_free[n & 1]), (n / 2 - 1) & 1, watch);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < D / 32; ++kk)
                        mma_ss_f8(tmem + (n & 1) * N, sdesc_sw(s_stage + st * C::kStage + 32 * kk, 16, sbo, C::kSwizzle),
                                  sdesc_sw(s_q + 32 * kk, 16, sbo, C::kSwizzle), idesc_s, kk > 0);
                    mma_commit(smem_u32(&sh.s_full[n & 1]));
                    if (g > w.g0) values(n - 1);
                }
            }
            if (ok && n > 0) values(n - 1);
        }
        __syncwarp();
    } else {
        // =================================================== weights and output
        const float ninf = __int_as_float(0xFF800000);
        const int group = warp / 4, gwarp = warp % 4, gtid = tid % 128;
        const int row0 = group * kRows;  // of the group's rows in the block
        const int row_blocks = p.units / p.Hkv;
        const uint32_t t_lane = (uint32_t)(gwarp * 32) << 16;
        constexpr uint32_t kNone = 0xFFFFFFFFu;
        uint32_t tmem = kNone;
        int n = 0;
        while (w.at < w.end) {
            paged_open<kKeys>(p, shape, sh.cost, w);
            if (w.g0 >= w.g1) continue;  // overhead alone (the same for every thread)
            const int len = w.len, seen = w.seen;
            const int head = w.h / row_blocks, block0 = (w.h - head * row_blocks) * RP, rows = min(RP, p.rows - block0);
            const long long out0 = ((long long)w.b * p.Hkv + head) * p.rows + block0;  // the block's first row of Q and O
            // ---- the queries' two parts; a warp per row, four elements a lane
            {
                const uint16_t* q = reinterpret_cast<const uint16_t*>(p.q) + out0 * D;
                uint2 v[kRows / 4];
#pragma unroll
                for (int i = 0; i < kRows / 4; ++i) {
                    const int row = row0 + gwarp + 4 * i;
                    v[i] = make_uint2(0, 0);
                    if (row < rows && lane < D / 4) v[i] = *reinterpret_cast<const uint2*>(q + (long long)row * D + 4 * lane);
                }
#pragma unroll
                for (int i = 0; i < kRows / 4; ++i) {
                    const int row = row0 + gwarp + 4 * i;
                    uint32_t big = __vmaxu2(v[i].x & 0x7FFF7FFFu, v[i].y & 0x7FFF7FFFu);  // as bits of a bf16
                    big = __reduce_max_sync(0xFFFFFFFFu, max(big & 0xFFFFu, big >> 16));
                    // exponent field f: the row is below 2^(f - 126), so below 2^8 once scaled by 2^(134 - f).  A row
                    // below 2^-100 is taken as zeros in part; one with an infinity or a NaN becomes NaN.
                    const int f = max((int)(big >> 7), 27);
                    const float down = f == 255 ? __int_as_float(0x7FFFFFFF) : __uint_as_float((uint32_t)(261 - f) << 23);
                    const float up = f == 255 ? __int_as_float(0x7FFFFFFF) : __uint_as_float((uint32_t)(f - 7) << 23);
                    uint32_t hi, lo;
                    split_e4m3(__uint_as_float(v[i].x << 16) * down, __uint_as_float(v[i].x & 0xFFFF0000u) * down,
                               __uint_as_float(v[i].y << 16) * down, __uint_as_float(v[i].y & 0xFFFF0000u) * down, hi, lo);
                    if (lane < D / 4) {
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            const int r = half * RP + row, chunk = lane / 4;
                            const int sw = D == 128 ? chunk ^ (r & 7) : chunk ^ ((r >> 1) & 3);
                            asm volatile("st.shared.u32 [%0], %1;" ::"r"(s_q + r * D + 16 * sw + 4 * (lane % 4)),
                                         "r"(half ? lo : hi)
                                         : "memory");
                        }
                    }
                    if (lane == 0) {
                        const int t = len - p.S_q + (block0 + row) % p.S_q;
                        sh.qs[row] = p.scale_log2 * up;
                        sh.last[row] = row >= rows ? -1 : p.causal ? t : len - 1;
                        sh.first[row] = p.window < 0 ? 0 : max(0, t - p.window);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sh.q_full));
                named_bar_sync(1 + group, 128);
            }
            if (tmem == kNone) tmem = tmem_ready();
            const uint32_t t_d = tmem + 2 * N;
            // positions every real row sees need no test: [all_from, all_to)
            const int all_to = p.causal ? len - p.S_q + 1 : len;
            const int all_from = p.window < 0 ? 0 : max(0, len - 1 - p.window);
            float acc[kRows], l[kRows], m[kRows], back[kRows];
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                acc[r] = l[r] = back[r] = 0.f;
                m[r] = 0.f;
            }
            unsigned unset = 0xFF;  // bit r: row r has seen no key yet, and m[r] is no reference
            // D^T of the tile before is added to the output
            auto add_values = [&](int tile) {
                wait(smem_u32(&sh.d_full), tile & 1, watch);
                __syncwarp();
                tc_fence_after();
                float hi[kRows], lo[kRows];
                load_parts<RP>(t_d + t_lane + row0, hi, lo);
#pragma unroll
                for (int r = 0; r < kRows; ++r) acc[r] = fmaf(fmaf(lo[r], 0.0625f, hi[r]), back[r], acc[r]);
            };
            for (int g = w.g0; g < w.g1; ++g, ++n) {
                const int st = n % kStages;
                const int first = (w.lo + g) * kKeys, pos = first + gtid;
                wait(smem_u32(&sh.s_full[n & 1]), (n / 2) & 1, watch);
                wait(full(st), (n / kStages) & 1, watch);  // seen by this thread too: it reads and clears what was loaded
                __syncwarp();
                tc_fence_after();
                const bool inside = pos >= seen && pos < len;
                const uint32_t sc = s_scale + st * C::kScale + 32 * (gtid / 16) + gtid % 16;
                const uint32_t ek = lds_u8(sc), ev = lds_u8(sc + 16);
                const float kf = exponent_factor(ek);
                const float kv = inside ? (float)((int)ev - 127) : -127.f;
                // scores in base 2, less the rows' references
                float x[kRows];
                {
                    float hi[kRows], lo[kRows];
                    load_parts<RP>(tmem + (n & 1) * N + t_lane + row0, hi, lo);
#pragma unroll
                    for (int r = 0; r < kRows; r += 4) {
                        const float4 q = *reinterpret_cast<const float4*>(&sh.qs[row0 + r]);
                        x[r] = fmaf(fmaf(lo[r], 0.0625f, hi[r]), kf * q.x, -m[r]);
                        x[r + 1] = fmaf(fmaf(lo[r + 1], 0.0625f, hi[r + 1]), kf * q.y, -m[r + 1]);
                        x[r + 2] = fmaf(fmaf(lo[r + 2], 0.0625f, hi[r + 2]), kf * q.z, -m[r + 2]);
                        x[r + 3] = fmaf(fmaf(lo[r + 3], 0.0625f, hi[r + 3]), kf * q.w, -m[r + 3]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sh.s_free[n & 1]));
                if (first < all_from || first + kKeys > all_to) {
#pragma unroll
                    for (int r = 0; r < kRows; r += 4) {  // (without branches: each would cost a wait for shared memory)
                        const int4 to = *reinterpret_cast<const int4*>(&sh.last[row0 + r]);
                        const int4 from = *reinterpret_cast<const int4*>(&sh.first[row0 + r]);
                        x[r] = !inside | (pos > to.x) | (pos < from.x) ? ninf : x[r];
                        x[r + 1] = !inside | (pos > to.y) | (pos < from.y) ? ninf : x[r + 1];
                        x[r + 2] = !inside | (pos > to.z) | (pos < from.z) ? ninf : x[r + 2];
                        x[r + 3] = !inside | (pos > to.w) | (pos < from.w) ? ninf : x[r + 3];
                    }
                }
                // ---- the tile's largest score of each row, and its largest value exponent
                {
                    float t[kRows];
#pragma unroll
                    for (int r = 0; r < kRows; ++r) t[r] = warp_max(x[r]);
                    const float kv_top = warp_max(kv);
                    if (lane == 0) {
                        float4* out = reinterpret_cast<float4*>(&sh.top[n & 1][gwarp][row0]);
                        out[0] = make_float4(t[0], t[1], t[2], t[3]);
                        out[1] = make_float4(t[4], t[5], t[6], t[7]);
                        sh.factor[n & 1][group][gwarp] = kv_top;
                    }
                }
                named_bar_sync(1 + group, 128);
                if (g > w.g0) add_values(n - 1);
                const float4 k4 = *reinterpret_cast<const float4*>(&sh.factor[n & 1][group][0]);
                const float k_top = fmaxf(fmaxf(k4.x, k4.y), fmaxf(k4.z, k4.w)) - 8.f;
                // what is the same for all positions is worked out once a warp, by lane r for row r, and handed round
                float top;
                {
                    const int r = row0 + lane % kRows;
                    top = fmaxf(fmaxf(sh.top[n & 1][0][r], sh.top[n & 1][1][r]),
                                fmaxf(sh.top[n & 1][2][r], sh.top[n & 1][3][r]));
                }
                // the reference moves when a score passes it by 2^16, and to a row's first score
                const bool fresh = unset >> (lane % kRows) & 1;
                const unsigned moved = __ballot_sync(0xFFFFFFFFu, fresh ? top > ninf : top > 16.f) & 0xFF;
                if (moved) {
#pragma unroll
                    for (int r = 0; r < kRows; ++r) {
                        const float by = moved >> r & 1 ? __shfl_sync(0xFFFFFFFFu, top, r) : 0.f;
                        const float fix = unset >> r & 1 ? 0.f : ex2(-by);
                        m[r] += by;
                        x[r] -= by;
                        acc[r] *= fix;
                        l[r] *= fix;
                    }
                    if (moved >> (lane % kRows) & 1) top = 0.f;
                    unset &= ~moved;
                }
                // weights of a tile 2^-100 below the reference count as zeros
                const bool far = !(top > -100.f);
                const float up_l = far ? 0.f : ex2(-top), back_l = far ? 0.f : ex2(top + k_top);
                const float kvf = ex2(kv - k_top);
                uint32_t hi[kRows / 2], lo[kRows / 2];
#pragma unroll
                for (int r = 0; r < kRows; r += 2) {
                    float y[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float e = ex2(x[r + i]);
                        l[r + i] += e;
                        y[i] = e * __shfl_sync(0xFFFFFFFFu, up_l, r + i) * kvf;
                        back[r + i] = __shfl_sync(0xFFFFFFFFu, back_l, r + i);
                    }
                    split2_e4m3(y[0], y[1], hi[r / 2], lo[r / 2]);
                }
                // column c of position t: 16 columns side by side, then the positions, then the next 16 columns
                const uint32_t at = s_p + 16 * gtid, ch = row0, cl = RP + row0;
                asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at + (ch / 16) * 16 * kKeys + ch % 16),
                             "r"(hi[0] | hi[1] << 16), "r"(hi[2] | hi[3] << 16)
                             : "memory");
                asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at + (cl / 16) * 16 * kKeys + cl % 16),
                             "r"(lo[0] | lo[1] << 16), "r"(lo[2] | lo[3] << 16)
                             : "memory");
                if (!inside && group == 0) {
                    // positions past the length or before the window may hold anything: weight zero times a NaN is a
                    // NaN, so their values become zero
                    const uint32_t v = s_stage + st * C::kStage + C::kTile + gtid * D;
#pragma unroll
                    for (int c = 0; c < D / 16; ++c)
                        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(v + 16 * c), "r"(0) : "memory");
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sh.p_full));
            }
            add_values(n - 1);
            tc_fence_before();
            // ---- the rows' sums over the threads, and the stretch's result.  The warp's sums, eight at once: each step halves
            // the rows that a lane still holds, until the lanes 4 r .. 4 r + 3 hold row r.
#pragma unroll
            for (int step = 0; step < 3; ++step) {
                const int o = 16 >> step, half = kRows / 2 >> step;
                const bool up = lane & o;
#pragma unroll
                for (int i = 0; i < half; ++i) {
                    const float give = up ? l[i] : l[i + half], keep = up ? l[i + half] : l[i];
                    l[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, o);
                }
            }
            l[0] += __shfl_xor_sync(0xFFFFFFFFu, l[0], 2);
            l[0] += __shfl_xor_sync(0xFFFFFFFFu, l[0], 1);
            if (lane % 4 == 0) sh.sum[gwarp][row0 + lane / 4] = l[0];
            named_bar_sync(1 + group, 128);
            const bool final = w.g0 == 0 && w.g1 == w.n;
            const long long slot = (2LL * blockIdx.x + (w.g0 > 0 ? 0 : 1)) * RP;
            // lane r works out what belongs to row r, for all threads
            const int mine = lane % kRows, my_row = row0 + mine;
            const float L = (sh.sum[0][my_row] + sh.sum[1][my_row]) + (sh.sum[2][my_row] + sh.sum[3][my_row]);
            const float inv = __frcp_rn(L);
            const unsigned none = __ballot_sync(0xFFFFFFFFu, L == 0.f);  // bit r: the row has seen nothing
            float out[kRows];
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                const float by = __shfl_sync(0xFFFFFFFFu, inv, r);
                out[r] = !final ? acc[r] : none >> r & 1 ? 0.f : acc[r] * by;
            }
            if (gtid < D) {
                if (final) {
                    __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(p.o) + (out0 + row0) * D + gtid;
#pragma unroll
                    for (int r = 0; r < kRows; ++r)
                        if (row0 + r < rows) o[r * D] = __float2bfloat16(out[r]);
                } else {
                    float* o = p.part_o + (slot + row0) * D + gtid;
#pragma unroll
                    for (int r = 0; r < kRows; ++r)
                        if (row0 + r < rows) __stcg(o + r * D, out[r]);
                }
            }
            if (gtid < kRows && my_row < rows) {
                float ref = m[0];
#pragma unroll
                for (int r = 1; r < kRows; ++r) ref = mine == r ? m[r] : ref;
                if (!final) __stcg(&p.part_ml[slot + my_row], make_float2(unset >> mine & 1 ? ninf : ref, L));
                else if (p.lse) p.lse[out0 + my_row] = (ref + log2f(L)) * 0.6931471805599453f;
            }
            if (w.g0 == 0 && tid == 0) paged_record_cut(p, cuts, shape, sh.cost, w, final);
            // before sh.sum, the queries and the row bounds are written again
            named_bar_sync(1 + group, 128);
        }
        if (tmem == kNone) tmem_ready();
    }
    // all warps meet behind their last copy and product
    __syncthreads();
    if (sh.abort) {
        drain();
        __syncthreads();
    }
    if (warp == kLoader + 1) {
        tc_fence_after();
        tmem_dealloc(sh.tmem, C::kCols);
    }
}

template <int D, int RP>
cudaError_t launch_rp(const PagedParams& p, int grid, cudaStream_t stream) {
    auto* f = paged_e4m3_kernel<D, RP>;
    cudaError_t e = smem_opt_in(reinterpret_cast<const void*>(f), Cfg<D, RP>::kSmem);
    if (e != cudaSuccess) return e;
    return launch_dependent(f, dim3((unsigned)grid), Cfg<D, RP>::kThreads, Cfg<D, RP>::kSmem, stream, p);
}
template <int D>
cudaError_t launch_d(const PagedParams& p, int grid, cudaStream_t stream) {
    switch (paged_rows_pad(p.rows, true)) {
        case 8: return launch_rp<D, 8>(p, grid, stream);
        case 16: return launch_rp<D, 16>(p, grid, stream);
        default: return launch_rp<D, 32>(p, grid, stream);
    }
}

}  // namespace

cudaError_t launch_paged_e4m3(const PagedParams& p, int grid, cudaStream_t stream) {
    return p.c.d == 64 ? launch_d<64>(p, grid, stream) : launch_d<128>(p, grid, stream);
}

}  // namespace attn
