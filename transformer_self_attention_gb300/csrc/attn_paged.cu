// Attention of a few new rows per sequence over a paged bf16 cache, and the joining of split sequences.
//
//     O_i = sum_j softmax_j(scale q_i . k_j) v_j over the cached positions j that row i sees.
//
// Bound by memory: every visible key and value row is read once per kv head, for 4 * rows flops per element
// read, rows = the query rows that share the kv head (up to 64).
//
// A persistent grid, two CTAs a multiprocessor, of four computing warps and up to four loading ones.  Lengths and page
// table are read on the device, so that a captured launch follows them: every CTA computes the same prefix sums of the
// lengths and takes its interval of the cost line (paged.h).  Inside a CTA the key blocks of a stretch (a CTA's part of
// a unit) go to the computing warps in turn.  Each warp, or each RW warps where there are more than 16 rows, has a ring
// of its own in shared memory, filled by a loading warp with one TMA box per 16 positions (keys and values of a head in
// one box, so that pages of any multiple of 16 work).  The warps share nothing until the stretch ends: each holds its own
// running maximum, sum and output tile (16 rows x d, fp32 registers).  Then their results are added through shared
// memory.  A unit cut between CTAs is joined by a second kernel, launched as a programmatic dependent, one to four warps
// a row; it adds the parts in their order, so that a result does not depend on who finishes first.  (Joined by the last CTA to
// arrive instead, 19 parts of 32 rows took 15 of a call's 44 us.)
//
// The products are m16n8k16 with fp32 accumulation: at the measured copy bandwidth an SM takes in 24 bytes a clock, 12
// elements, 188 multiply-adds at 16 rows of the 1024 these products do a clock.  Up to 32 rows a weight enters the
// second product as the sum of two bf16 numbers (2^-16 of it at most is lost; 1.5% of the time at 8 rows, 141 us for 904
// MB), above that, where these products are the limit, as one (2^-8; two took 143 us for 452 MB at 64 rows
// against 110).  The weights' sum is taken before.
#include <cuda_bf16.h>

#include <algorithm>
#include <cstddef>
#include <type_traits>

#include "device_once.h"
#include "paged_device.h"

namespace attn {

using namespace ptx;

namespace {

constexpr int kWarps = 4;                       // computing warps of a CTA
constexpr int kThreads = 64 * kWarps;           // and a warpgroup of which one warp loads
// Registers: 128 a thread at launch (two CTAs of 256 threads); the loading warpgroup hands its share over.
constexpr int kLoadRegs = 40, kComputeRegs = 216;
static_assert((kLoadRegs + kComputeRegs) * 32 * kWarps <= 128 * kThreads, "the split fits what the block was launched with");
constexpr int kCtasPerSm = 2;
constexpr int kRingBytes = 96 * 1024;           // of all rings of a CTA

template <int D>
struct Cfg {
    static constexpr int kParts = D * 2 / 128;                     // of a row, 128 bytes each in shared memory
    static constexpr int kBoxBytes = 2 * 16 * D * 2;               // keys and values of 16 positions
    static constexpr int kKeys = paged_shape(D, false).keys;       // positions of a key block
    static constexpr int kBoxes = kKeys / 16;
    static constexpr int kBlockBytes = kBoxes * kBoxBytes;
};
template <int D, int RW>
struct Ring {
    static constexpr int kRings = kWarps / RW;
    static constexpr int kStages = kRingBytes / kRings / Cfg<D>::kBlockBytes;
    static constexpr int kBytes = kRings * kStages * Cfg<D>::kBlockBytes;
};

__device__ __forceinline__ void tma_load_box(uint32_t dst, const CUtensorMap* map, uint32_t bar, int slot, int unit) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(slot), "r"(0), "r"(0), "r"(unit), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void ldm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The joining of the warps' results takes the output in passes of COLS columns and ROWS rows a warp.
template <int ROWS>
struct Red {
    static constexpr int kCols = 512 / ROWS;  // 64 columns of 8 rows, 32 of 16
    static constexpr int kPitch = kCols + 4;
};

// Shared memory of a CTA besides the rings (behind them).
struct Shared {
    unsigned cost[kPagedMaxBatch + 4];   // cost of the sequences before b, for one kv head
    alignas(16) float red[kWarps * 16 * Red<16>::kPitch];  // read as float4
    float2 ml[kWarps * 16];
    unsigned long long full[12 * kWarps], empty[12 * kWarps];
    unsigned scan[2 * kWarps];
    int abort;
};
static_assert(offsetof(Shared, red) % 16 == 0 && offsetof(Shared, full) % 8 == 0 && offsetof(Shared, ml) % 8 == 0 &&
                  alignof(Shared) == 16 && Red<8>::kPitch * 8 <= Red<16>::kPitch * 16,
              "alignment of the shared accesses, room for either pass");

template <int D, int RW>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) paged_kernel(const __grid_constant__ PagedParams p) {
    using C = Cfg<D>;
    using R = Ring<D, RW>;
    constexpr PagedShape shape = paged_shape(D, false);
    constexpr int kRings = R::kRings, kStages = R::kStages;
    static_assert(kRings * kStages <= 12 * kWarps, "barriers");
    extern __shared__ uint8_t smem_raw[];
    // boxes are swizzled by address: the rings begin on a 1024-byte boundary
    uint8_t* const ring_base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    Shared& sh = *reinterpret_cast<Shared*>(ring_base + R::kBytes);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int Hkv = p.Hkv, S_q = p.S_q, window = p.window;

    if (tid < kRings * kStages) {
        mbar_init(smem_u32(&sh.full[tid]), 1);
        mbar_init(smem_u32(&sh.empty[tid]), RW);
    }
    if (tid == 0) {
        prefetch_tmap(&p.tm);
        sh.abort = 0;
    }
    fence_barrier_init();
    wait_for_kernel_before();
    int busy;
    const unsigned W = paged_prefix<C::kKeys, kThreads>(p, shape, sh.cost, sh.scan, busy) * p.units;
    const PagedCuts cuts(W, busy * p.units, gridDim.x, shape);
    let_kernel_behind_in();
    if (busy < p.B) paged_empty_rows<D, kThreads>(p, sh.cost);
    if (tid == 0 && !p.by_unit) p.cut[blockIdx.x] = make_int2(-1, 0);
    if (blockIdx.x >= cuts.C || W == 0) return;
    const Watch watch{&sh.abort, p.c.err, p.watchdog_ns};
    Walk w = paged_begin(p, cuts, sh.cost);
    const uint32_t ring_smem0 = smem_u32(ring_base);
    // The end of every warp: all meet behind their last copy, and after a wait that ran out those still on their way are
    // waited for before the CTA gives its shared memory up.
    auto finish = [&]() {
        named_bar_sync(2, kThreads);
        if (*watch.abort) drain();
    };

    // =================================================== the loading warps: one for each ring
    if (warp >= kWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLoadRegs));
        const int ring = warp - kWarps;
        if (ring >= kRings) {
            finish();
            return;
        }
        const uint32_t dst0 = ring_smem0 + ring * kStages * C::kBlockBytes;
        const uint32_t full0 = smem_u32(&sh.full[ring * kStages]), empty0 = smem_u32(&sh.empty[ring * kStages]);
        int g = 0;  // next block of the ring in the stretch
        // A batch: up to 32 blocks of the ring in one stretch, a lane each.  The next batch's page numbers are on their
        // way while this one's blocks are issued.
        struct Batch {
            int n;
            int unit[C::kBoxes], slot[C::kBoxes];  // page * Hkv + head, -1: the box is not needed
        };
        auto fetch = [&](Batch& f) {
            f.n = 0;
            while (g >= w.g1) {
                if (w.at >= w.end) return;
                paged_open<C::kKeys>(p, shape, sh.cost, w);
                g = w.g0 + ring;
            }
            f.n = min(32, (w.g1 - g + kRings - 1) / kRings);
            const int first = (w.lo + g + lane * kRings) * C::kKeys;
#pragma unroll
            for (int k = 0; k < C::kBoxes; ++k) {
                const int pos = first + 16 * k;
                f.unit[k] = -1;
                if (lane >= f.n || pos >= w.len || pos + 16 <= w.seen) continue;
                const int index = (unsigned)pos / (unsigned)p.c.page;
                f.slot[k] = pos - index * p.c.page;
                int page = p.t.pages[w.b * p.t.stride + index];
                if (page < 0 || page >= p.c.n_pages) {
                    atomicOr(p.c.err, kCacheErrPage);
                    page = 0;
                }
                f.unit[k] = page * Hkv + w.h;
            }
            g += 32 * kRings;
        };
        int fill = 0;
        uint32_t parity = 1;  // of the slot's last emptying; the first round finds every slot empty
        Batch now, then;
        fetch(now);
        while (now.n) {
            fetch(then);
            for (int i = 0; i < now.n; ++i) {
                if (!__all_sync(0xFFFFFFFFu, i + 1 != p.withhold && wait(empty0 + 8 * fill, parity, watch))) {
                    then.n = 0;
                    break;
                }
                const uint32_t bar = full0 + 8 * fill;
                int unit[C::kBoxes], slot[C::kBoxes], boxes = 0;
#pragma unroll
                for (int k = 0; k < C::kBoxes; ++k) {
                    unit[k] = __shfl_sync(0xFFFFFFFFu, now.unit[k], i);
                    slot[k] = __shfl_sync(0xFFFFFFFFu, now.slot[k], i);
                    boxes += unit[k] >= 0;
                }
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar, boxes * C::kBoxBytes);
#pragma unroll
                    for (int k = 0; k < C::kBoxes; ++k) {
                        if (unit[k] >= 0)
                            tma_load_box(dst0 + fill * C::kBlockBytes + k * C::kBoxBytes, &p.tm, bar, slot[k], unit[k]);
                    }
                }
                if (++fill == kStages) {
                    fill = 0;
                    parity ^= 1;
                }
            }
            now = then;
        }
        finish();
        return;
    }

    // =================================================== the computing warps
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kComputeRegs));
    const int ring = warp / RW, rw = warp % RW;
    const int quad = lane / 4, pair = lane % 4;
    const uint32_t ring_smem = ring_smem0 + ring * kStages * C::kBlockBytes;
    const uint32_t full = smem_u32(&sh.full[ring * kStages]), empty = smem_u32(&sh.empty[ring * kStages]);
    const float ninf = __int_as_float(0xFF800000);
    constexpr int kTiles = C::kKeys / 8;  // score tiles of a block
    // A wait ran out: the warp takes no further block and frees no place, so that its loading warp stops too; it goes on
    // to the ends of the stretches, where the warps meet.  The outputs are undefined.
    bool dead = false;
    int stage = 0;
    uint32_t phase = 0;
    while (w.at < w.end) {
        paged_open<C::kKeys>(p, shape, sh.cost, w);
        if (w.g0 >= w.g1) continue;  // overhead alone (the same for every warp of the CTA)
        const int len = w.len, seen = w.seen;
        const int row0 = 16 * rw;
        // rows quad and quad + 8 of the warp's 16: their last and first visible position
        int last[2], first_seen[2];
        uint32_t qf[D / 16][4];  // the queries as the first operand
        {
            const uint16_t* q =
                reinterpret_cast<const uint16_t*>(p.q) + ((long long)w.b * Hkv + w.h) * p.rows * D;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = row0 + quad + 8 * r;
                const bool real = row < p.rows;
                const int t = len - S_q + row % S_q;
                last[r] = !real ? -1 : p.causal ? t : len - 1;
                first_seen[r] = window < 0 ? 0 : max(0, t - window);
                const uint16_t* qr = q + (long long)row * D;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    qf[ks][r] = real ? *reinterpret_cast<const uint32_t*>(qr + 16 * ks + 2 * pair) : 0u;
                    qf[ks][2 + r] = real ? *reinterpret_cast<const uint32_t*>(qr + 16 * ks + 8 + 2 * pair) : 0u;
                }
            }
        }
        // positions every real row sees need no test: [all_from, all_to)
        const int all_to = p.causal ? len - S_q + 1 : len;
        const int all_from = window < 0 ? 0 : max(0, len - 1 - window);
        float acc[D / 8][4];
#pragma unroll
        for (int j = 0; j < D / 8; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
        float m[2] = {ninf, ninf}, l[2] = {0.f, 0.f};

        for (int g = w.g0 + ring; g < w.g1 && !dead; g += kRings) {
            const int first = (w.lo + g) * C::kKeys;
            const uint32_t buf = ring_smem + stage * C::kBlockBytes;
            if (!__all_sync(0xFFFFFFFFu, wait(full + 8 * stage, phase, watch))) {
                dead = true;
                break;
            }
            if (first + C::kKeys > len || first < seen) {
                // positions past the length or before the window may hold anything: weight zero times a NaN is a
                // NaN, so their values become zero (their scores are masked below)
#pragma unroll 1
                for (int key = 0; key < C::kKeys; ++key) {
                    if (first + key >= seen && first + key < len) continue;
                    const uint32_t v = buf + (key / 16) * C::kBoxBytes + C::kBoxBytes / 2 + (key % 16) * 128;
                    if (lane < 8 * C::kParts) {
                        const uint32_t at = v + (lane / 8) * 16 * 128 + (lane % 8) * 16;
                        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0) : "memory");
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
            }
            // ---- S = Q K^T, in base 2
            float s[kTiles][4];
            {
                // two chains a tile: a product waits 20 clocks for the one before
                float s2[kTiles][4];
#pragma unroll
                for (int j = 0; j < kTiles; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[j][i] = s2[j][i] = 0.f;
#pragma unroll
                for (int bx = 0; bx < C::kBoxes; ++bx) {
                    // one x4 load: keys 0-7 and 8-15, 16 elements of the row (one step)
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        const int row = lane % 8 + 8 * (lane / 16), chunk = (2 * ks + (lane / 8 & 1)) % 8;
                        uint32_t r[4];
                        ldm4(r, buf + bx * C::kBoxBytes + (ks / 4) * 16 * 128 + row * 128 +
                                    (chunk ^ (row & 7)) * 16);
                        if (ks % 2) {
                            mma_bf16(s2[2 * bx], qf[ks], r[0], r[1]);
                            mma_bf16(s2[2 * bx + 1], qf[ks], r[2], r[3]);
                        } else {
                            mma_bf16(s[2 * bx], qf[ks], r[0], r[1]);
                            mma_bf16(s[2 * bx + 1], qf[ks], r[2], r[3]);
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < kTiles; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[j][i] = (s[j][i] + s2[j][i]) * p.scale_log2;
            }
            if (first < all_from || first + C::kKeys > all_to) {
#pragma unroll
                for (int j = 0; j < kTiles; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int pos = first + 8 * j + 2 * pair + (i & 1);
                        if (pos > last[i >> 1] || pos < first_seen[i >> 1]) s[j][i] = ninf;
                    }
            }
            // ---- the reference of the weights: any number near the running maximum serves (sums are float32 and bf16
            // has its range), so it moves, for all rows together, only when a score passes it by 2^16
            float top[2] = {s[0][0], s[0][2]};
#pragma unroll
            for (int j = 0; j < kTiles; ++j) {
                top[0] = fmax3(top[0], s[j][0], s[j][1]);
                top[1] = fmax3(top[1], s[j][2], s[j][3]);
            }
            if (__any_sync(0xFFFFFFFFu, top[0] > m[0] + 16.f || top[1] > m[1] + 16.f)) {
                float fix[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float t = fmaxf(top[r], __shfl_xor_sync(0xFFFFFFFFu, top[r], 1));
                    t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, 2));
                    const float to = fmaxf(t, m[r]);
                    fix[r] = to == m[r] ? 1.f : ex2(m[r] - to);
                    m[r] = to;
                    l[r] *= fix[r];
                }
#pragma unroll
                for (int j = 0; j < D / 8; ++j) {
                    acc[j][0] *= fix[0];
                    acc[j][1] *= fix[0];
                    acc[j][2] *= fix[1];
                    acc[j][3] *= fix[1];
                }
            }
            const float base[2] = {m[0] == ninf ? 0.f : m[0], m[1] == ninf ? 0.f : m[1]};
            {
                constexpr bool kTwoParts = RW <= 2;
                uint32_t pf[C::kBoxes][4], pl[C::kBoxes][4];
#pragma unroll
                for (int j = 0; j < kTiles; ++j) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        s[j][i] = ex2(s[j][i] - base[i >> 1]);
                        l[i >> 1] += s[j][i];
                    }
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const uint32_t h = pack_bf16x2(s[j][2 * r], s[j][2 * r + 1]);
                        pf[j / 2][2 * (j % 2) + r] = h;
                        if (kTwoParts)
                            pl[j / 2][2 * (j % 2) + r] = pack_bf16x2(s[j][2 * r] - __uint_as_float(h << 16),
                                                                     s[j][2 * r + 1] - __uint_as_float(h & 0xFFFF0000u));
                    }
                }
#pragma unroll
                for (int bx = 0; bx < C::kBoxes; ++bx) {
#pragma unroll
                    for (int c2 = 0; c2 < D / 16; ++c2) {
                        const int row = lane % 16, chunk = (2 * c2 + lane / 16) % 8;
                        uint32_t r[4];
                        ldm4t(r, buf + bx * C::kBoxBytes + C::kBoxBytes / 2 + (c2 / 4) * 16 * 128 + row * 128 +
                                     (chunk ^ (row & 7)) * 16);
                        mma_bf16(acc[2 * c2], pf[bx], r[0], r[1]);
                        mma_bf16(acc[2 * c2 + 1], pf[bx], r[2], r[3]);
                        if (kTwoParts) {
                            mma_bf16(acc[2 * c2], pl[bx], r[0], r[1]);
                            mma_bf16(acc[2 * c2 + 1], pl[bx], r[2], r[3]);
                        }
                    }
                }
            }
            // the block is read: its place is free
            __syncwarp();
            if (lane == 0) mbar_arrive(empty + 8 * stage);
            stage = stage + 1 == kStages ? 0 : stage + 1;
            if (stage == 0) phase ^= 1;
        }

        // ---- the warps' results of this stretch, added
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 1);
            l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 2);
            if (pair == 0) sh.ml[warp * 16 + quad + 8 * r] = make_float2(m[r], l[r]);
        }
        named_bar_sync(1, 32 * kWarps);
        // row `row` of the unit: the maximum over the rings, and the sum
        auto row_ml = [&](int row) {
            float M = ninf, L = 0.f;
#pragma unroll
            for (int g = 0; g < kRings; ++g) M = fmaxf(M, sh.ml[(g * RW + row / 16) * 16 + row % 16].x);
#pragma unroll
            for (int g = 0; g < kRings; ++g) {
                const float2 v = sh.ml[(g * RW + row / 16) * 16 + row % 16];
                L += v.x == ninf ? v.y : v.y * ex2(v.x - M);
            }
            return make_float2(M, L);
        };
        float fix[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) fix[r] = m[r] == ninf ? 0.f : ex2(m[r] - row_ml(row0 + quad + 8 * r).x);
        const bool final = w.g0 == 0 && w.g1 == w.n;
        const int unit = w.b * Hkv + w.h;
        const int slot = 2 * blockIdx.x + (w.g0 > 0 ? 0 : 1);
        constexpr int kRowsPad = 16 * RW;
        float* part = p.part_o + (long long)slot * kRowsPad * D;
        auto add = [&](auto rows_const) {
            constexpr int ROWS = decltype(rows_const)::value, COLS = Red<ROWS>::kCols, PITCH = Red<ROWS>::kPitch;
            constexpr int STEP = COLS < D ? COLS : D;
#pragma unroll
            for (int c0 = 0; c0 < D; c0 += STEP) {
                float* mine = sh.red + warp * ROWS * PITCH;
                if (c0) named_bar_sync(1, 32 * kWarps);
#pragma unroll
                for (int r = 0; r < ROWS / 8; ++r)
#pragma unroll
                    for (int jj = 0; jj < STEP / 8; ++jj)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int col = 8 * jj + 2 * pair + i;
                            mine[(quad + 8 * r) * PITCH + col] = acc[c0 / 8 + jj][2 * r + i] * fix[r];
                        }
                named_bar_sync(1, 32 * kWarps);
#pragma unroll
                for (int x = tid; x < ROWS * RW * STEP / 4; x += 32 * kWarps) {
                    const int row = x / (STEP / 4), c4 = x % (STEP / 4) * 4;
                    if (row >= p.rows) continue;
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int g = 0; g < kRings; ++g) {
                        const float4 y = *reinterpret_cast<const float4*>(
                            &sh.red[((g * RW + row / ROWS) * ROWS + row % ROWS) * PITCH + c4]);
                        v.x += y.x; v.y += y.y; v.z += y.z; v.w += y.w;
                    }
                    if (final) {
                        const float L = row_ml(row).y;
                        const float inv = L == 0.f ? 0.f : 1.f / L;
                        const uint2 o = make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
                        *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p.o) +
                                                  ((long long)unit * p.rows + row) * D + c0 + c4) = o;
                    } else {
                        __stcg(reinterpret_cast<float4*>(part + row * D + c0 + c4), v);
                    }
                }
            }
        };
        if (RW == 1 && p.rows <= 8) add(std::integral_constant<int, 8>{});
        else add(std::integral_constant<int, 16>{});
        if (tid < p.rows) {
            const float2 v = row_ml(tid);
            if (!final) __stcg(&p.part_ml[slot * kRowsPad + tid], v);
            else if (p.lse) p.lse[(long long)unit * p.rows + tid] = (v.x + log2f(v.y)) * 0.6931471805599453f;
        }
        if (w.g0 == 0 && tid == 0) paged_record_cut(p, cuts, shape, sh.cost, w, final);
        named_bar_sync(1, 32 * kWarps);  // sh.ml and sh.red are free again
    }
    finish();
}

// Joins the parts of one cut unit: O = sum_k 2^(m_k - M) O_k / L with M = max m_k, L = sum_k 2^(m_k - M) l_k.  The first
// part is in its CTA's second slot (the unit begins inside the interval), the others in their CTA's first.  SPLIT warps a
// row, a stretch of the parts each: four where a unit has eight parts or more, two from three parts on, else one.  What
// counts is the chain of round trips to L2 (what is cut; then maxima, sums and parts together), and that the blocks fit
// on the chip at once.  16 sequences of 19 parts of 32 rows: 26.6 us a decode step, 29.4 with one warp a row that reads
// the parts behind the maxima; 64 units of 5 parts of 16 rows: 26.5 us with two warps a row, 27.6 with four.
constexpr int kMergeWarps = 8;
template <int D, int SPLIT>
__global__ void __launch_bounds__(32 * kMergeWarps) paged_merge_kernel(const __grid_constant__ PagedParams p, int rows_pad) {
    constexpr int kVec = D / 32, kBatch = SPLIT == 1 ? 16 : 8, kRows = kMergeWarps / SPLIT;
    __shared__ float sums[SPLIT == 1 ? 1 : kMergeWarps][SPLIT == 1 ? 1 : D];
    __shared__ float weights[SPLIT == 1 ? 1 : kMergeWarps];
    wait_for_kernel_before();
    let_kernel_behind_in();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, share = warp % SPLIT;
    const int row = blockIdx.y * kRows + warp / SPLIT;
    const int2 cut = __ldcg(&p.cut[blockIdx.x]);
    if (cut.x < 0) return;
    const int unit = p.by_unit ? (int)blockIdx.x : cut.x, k0 = p.by_unit ? cut.x : (int)blockIdx.x;
    const int blocks = p.units / p.Hkv, head = unit / blocks, row_block = unit - head * blocks;
    const int out_row = row_block * rows_pad + row;
    const bool live = row < rows_pad && out_row < p.rows;
    if (SPLIT == 1 && !live) return;
    const int n = live ? cut.y - k0 + 1 : 0, lo = n * share / SPLIT, hi = n * (share + 1) / SPLIT;  // parts of the warp
    const float ninf = __int_as_float(0xFF800000);
    auto at = [&](int i) { return (long long)(2 * (k0 + i) + (i == 0)) * rows_pad + row; };
    float y[kBatch][kVec];
    auto load = [&](int first) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (first + i >= hi) continue;
            const float* src = p.part_o + at(first + i) * D;
            if constexpr (D == 128) {
                const float4 t = __ldcg(reinterpret_cast<const float4*>(src) + lane);
                y[i][0] = t.x; y[i][1] = t.y; y[i][kVec - 2] = t.z; y[i][kVec - 1] = t.w;
            } else {
                const float2 t = __ldcg(reinterpret_cast<const float2*>(src) + lane);
                y[i][0] = t.x; y[i][1] = t.y;
            }
        }
    };
    load(lo);
    float M = ninf, L = 0.f, v[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) v[i] = 0.f;
    for (int i = lane; i < n; i += 32) M = fmaxf(M, __ldcg(&p.part_ml[at(i)]).x);
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
    for (int first = lo; first < hi; first += kBatch) {
        if (first > lo) load(first);
        float f = 0.f;
        if (lane < kBatch && first + lane < hi) {
            const float2 t = __ldcg(&p.part_ml[at(first + lane)]);
            // a part without a maximum has seen nothing (sum 0), or only NaN
            f = t.x == ninf ? t.y : ex2(t.x - M);
            L += t.x == ninf ? t.y : t.y * f;
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const float fi = __shfl_sync(0xFFFFFFFFu, f, i);
            if (first + i >= hi) continue;
#pragma unroll
            for (int j = 0; j < kVec; ++j) v[j] += fi * y[i][j];
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xFFFFFFFFu, L, o);
    if constexpr (SPLIT > 1) {
#pragma unroll
        for (int j = 0; j < kVec; ++j) sums[warp][kVec * lane + j] = v[j];
        if (lane == 0) weights[warp] = L;
        __syncthreads();
        if (share || !live) return;
#pragma unroll
        for (int w = 1; w < SPLIT; ++w) {
            L += weights[warp + w];
#pragma unroll
            for (int j = 0; j < kVec; ++j) v[j] += sums[warp + w][kVec * lane + j];
        }
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const long long out = (long long)head * p.rows + out_row;
    uint32_t* o = reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(p.o) + out * D) + lane * (D / 64);
#pragma unroll
    for (int i = 0; i < D / 64; ++i) o[i] = pack_bf16x2(v[2 * i] * inv, v[2 * i + 1] * inv);
    if (p.lse && lane == 0) p.lse[out] = (M + log2f(L)) * 0.6931471805599453f;
}

template <int D, int RW>
cudaError_t launch_rw(const PagedParams& p, int grid, cudaStream_t stream) {
    constexpr int smem = 1024 + Ring<D, RW>::kBytes + (int)sizeof(Shared);
    static_assert(smem <= 115712, "two CTAs per multiprocessor");
    auto* f = paged_kernel<D, RW>;
    cudaError_t e = smem_opt_in(reinterpret_cast<const void*>(f), smem);
    if (e != cudaSuccess) return e;
    return launch_dependent(f, dim3((unsigned)grid), kThreads, smem, stream, p);
}
template <int D>
cudaError_t launch_d(const PagedParams& p, int grid, cudaStream_t stream) {
    switch (paged_rows_pad(p.rows, false)) {
        case 16: return launch_rw<D, 1>(p, grid, stream);
        case 32: return launch_rw<D, 2>(p, grid, stream);
        default: return launch_rw<D, 4>(p, grid, stream);
    }
}

}  // namespace

int paged_rows_pad(int rows, bool e4m3) {
    return e4m3 && rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 || e4m3 ? 32 : 64;
}
int paged_row_blocks(int rows, bool e4m3) { return e4m3 && rows > 32 ? 2 : 1; }
int paged_ctas_per_sm(int rows, bool e4m3) { return !e4m3 || rows <= 16 ? 2 : 1; }

cudaError_t launch_paged_bf16(const PagedParams& p, int grid, cudaStream_t stream) {
    return p.c.d == 64 ? launch_d<64>(p, grid, stream) : launch_d<128>(p, grid, stream);
}

cudaError_t launch_paged_merge(const PagedParams& p, int grid, int rows_pad, cudaStream_t stream) {
    const int units = p.by_unit ? p.B * p.units : grid, parts = grid / units, rows = std::min(p.rows, rows_pad);
    const int split = parts >= 8 ? 4 : parts >= 3 ? 2 : 1, per = kMergeWarps / split;
    const dim3 blocks((unsigned)units, (unsigned)((rows + per - 1) / per));
    auto go = [&](auto* f) { return launch_dependent(f, blocks, 32 * kMergeWarps, 0, stream, p, rows_pad); };
    if (p.c.d == 64)
        return split == 4 ? go(paged_merge_kernel<64, 4>)
                          : split == 2 ? go(paged_merge_kernel<64, 2>) : go(paged_merge_kernel<64, 1>);
    return split == 4 ? go(paged_merge_kernel<128, 4>)
                      : split == 2 ? go(paged_merge_kernel<128, 2>) : go(paged_merge_kernel<128, 1>);
}

}  // namespace attn
