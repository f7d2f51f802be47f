// Attention of a few new rows per sequence over a paged cache (bf16 or E4M3).
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
// memory.  A unit cut between CTAs is joined by a second kernel, launched as a programmatic dependent, a warp per row;
// it adds the parts in their order, so that a result does not depend on who finishes first.
//
// bf16 caches use m16n8k16 products: at the measured copy bandwidth an SM takes in 24 bytes a clock, 12 elements, 188
// multiply-adds at 16 rows of the 1024 these products do a clock.  P is rounded to bf16 for the second product (2^-8 of a
// weight at most); its sum is taken before.  E4M3 caches use m16n8k32 products on the codes as they are, with the other
// operand, Q or P, as the sum of two E4M3 numbers (8 significant bits, all of a bf16 number's).  Turning the codes into
// bf16 first cost 1260 instructions a block of 32 positions instead of about 450, and each bf16 product takes 8 clocks a
// scheduler against 4.3 for one of twice the depth.
#include <cuda_bf16.h>

#include <algorithm>
#include <cstddef>
#include <type_traits>

#include "device_once.h"
#include "paged.h"
#include "sm103_ptx.h"

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

template <int D, bool E4M3>
struct Cfg {
    static constexpr int kRowBytes = D * (E4M3 ? 1 : 2);
    static constexpr int kInner = kRowBytes < 128 ? kRowBytes : 128;  // bytes of a row part in shared memory
    static constexpr int kBoxBytes = 2 * 16 * kRowBytes;              // keys and values of 16 positions
    static constexpr int kBoxes = E4M3 || kBoxBytes < 8192 ? 2 : 1;   // an E4M3 product spans 32 positions
    static constexpr int kKeys = 16 * kBoxes;                         // positions of a key block
    static constexpr int kBlockBytes = kBoxes * kBoxBytes;
    static constexpr int kScaleBytes = E4M3 ? 32 * kBoxes : 0;
    static_assert(kBoxBytes % 1024 == 0 && kScaleBytes % 16 == 0, "alignment of boxes and of what follows the rings");
};
template <int D, bool E4M3, int RW>
struct Ring {
    using C = Cfg<D, E4M3>;
    static constexpr int kRings = kWarps / RW;
    static constexpr int kStages = kRingBytes / kRings / C::kBlockBytes;
    static constexpr int kBytes = kRings * kStages * (C::kBlockBytes + C::kScaleBytes);
};

__device__ __forceinline__ void tma_load_box(uint32_t dst, const CUtensorMap* map, uint32_t bar, int slot, int unit) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(slot), "r"(0), "r"(0), "r"(unit), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
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
__device__ __forceinline__ void mma_e4m3(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The same from zero.
__device__ __forceinline__ void mma_e4m3_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// Four floats of magnitude at most 448 as two E4M3 numbers each: x = hi + part * lo, with part a power of two and the
// remainder taken exactly.  hi rounds to four significant bits, so lo holds four more (down to the smallest step).
__device__ __forceinline__ void split_e4m3(float x0, float x1, float x2, float x3, float inv_part, uint32_t& hi,
                                           uint32_t& lo) {
    hi = pack_e4m3x4(x0, x1, x2, x3);
    uint32_t h01, h23;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h01) : "h"((uint16_t)hi));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h23) : "h"((uint16_t)(hi >> 16)));
    float f0, f1, f2, f3;
    asm("{.reg .f16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b;}" : "=f"(f0), "=f"(f1) : "r"(h01));
    asm("{.reg .f16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b;}" : "=f"(f2), "=f"(f3) : "r"(h23));
    lo = pack_e4m3x4((x0 - f0) * inv_part, (x1 - f1) * inv_part, (x2 - f2) * inv_part, (x3 - f3) * inv_part);
}
__device__ __forceinline__ float exponent_factor(uint32_t e) {  // 2^(e - 127); e = 255 (NaN codes beside it): inf
    return __uint_as_float(max(e << 23, 0x00400000u));
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t addr) {
    uint16_t e;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(e) : "r"(addr) : "memory");
    return e;
}

// Where a warp (or a loading lane) stands in its CTA's interval of the cost line.
struct Walk {
    unsigned at, end;   // cost positions
    int b, h, n;        // current unit and its key blocks
    int g, g1;          // blocks [g, g1) of the stretch still to take (g advances by the number of rings)
    int g0;             // first block of the stretch
    int lo;             // first key block of the sequence
    int len, seen;      // its visible positions: [seen, len)
};

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
};
static_assert(offsetof(Shared, red) % 16 == 0 && offsetof(Shared, full) % 8 == 0 && offsetof(Shared, ml) % 8 == 0 &&
                  alignof(Shared) == 16 && Red<8>::kPitch * 8 <= Red<16>::kPitch * 16,
              "alignment of the shared accesses, room for either pass");

template <int D, bool E4M3, int RW>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) paged_kernel(const __grid_constant__ PagedParams p) {
    using C = Cfg<D, E4M3>;
    using R = Ring<D, E4M3, RW>;
    constexpr int kRings = R::kRings, kStages = R::kStages;
    static_assert(kRings * kStages <= 12 * kWarps, "barriers");
    extern __shared__ uint8_t smem_raw[];
    // boxes are swizzled by address: the rings begin on a 1024-byte boundary
    uint8_t* const ring_base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    Shared& sh = *reinterpret_cast<Shared*>(ring_base + R::kBytes);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int Hkv = p.Hkv, S_q = p.S_q, window = p.window;

    // ---- prefix sums of the sequences' cost, of one kv head (the host keeps the whole below 2^31)
    const int room = p.t.max_pages * p.c.page;
    auto blocks_of = [&](int n, int& lo) {
        if (n < 0 || n > room) n = 0;
        int hi;
        paged_blocks(n, S_q, window, C::kKeys, lo, hi);
        return hi - lo;
    };
    if (tid < kRings * kStages) {
        mbar_init(smem_u32(&sh.full[tid]), 1);
        mbar_init(smem_u32(&sh.empty[tid]), RW);
    }
    if (tid == 0) {
        prefetch_tmap(&p.tm);
        sh.cost[0] = 0;
    }
    fence_barrier_init();
    unsigned carry = 0;
    int busy = 0;  // sequences with keys
    for (int b0 = 0; b0 < p.B; b0 += kThreads) {
        const int b = b0 + tid;
        unsigned x = 0;
        if (b < p.B) {
            const int len = p.t.len[b];
            int lo;
            const int n = blocks_of(len, lo);
            x = paged_cost(n);
            if (blockIdx.x == 0 && (len < 0 || len > room)) atomicOr(p.c.err, kCacheErrPosition);
        }
        const bool some = x != 0;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const unsigned y = __shfl_up_sync(0xFFFFFFFFu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) sh.scan[warp] = x;
        busy += __syncthreads_count(some);
        unsigned before = carry, all = carry;
#pragma unroll
        for (int w = 0; w < 2 * kWarps; ++w) {
            if (w < warp) before += sh.scan[w];
            all += sh.scan[w];
        }
        if (b < p.B) sh.cost[b + 1] = before + x;
        carry = all;
        __syncthreads();
    }
    const unsigned W = carry * Hkv;
    const PagedCuts cuts(W, busy * Hkv, gridDim.x);
    // the joining kernel may be scheduled from here on: it waits for this grid before it reads anything
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // ---- sequences without keys: rows of zeros, LSE -inf
    if (busy < p.B) {
        for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
            if (sh.cost[b + 1] != sh.cost[b]) continue;
            uint4* o = reinterpret_cast<uint4*>(p.o) + (long long)b * p.Hq * S_q * (D / 8);
            for (int i = tid; i < p.Hq * S_q * (D / 8); i += kThreads) o[i] = make_uint4(0, 0, 0, 0);
            if (p.lse)
                for (int i = tid; i < p.Hq * S_q; i += kThreads)
                    p.lse[(long long)b * p.Hq * S_q + i] = __int_as_float(0xFF800000);
        }
    }
    if (tid == 0) p.cut[blockIdx.x] = make_int2(-1, 0);
    if (blockIdx.x >= cuts.C || W == 0) return;

    // ---- the CTA's interval
    Walk w;
    w.at = cuts.begin(blockIdx.x);
    w.end = cuts.begin(blockIdx.x + 1);
    {
        int lo = 0, hi = p.B - 1;  // the last b whose cost begins at or before w.at
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (sh.cost[mid] * Hkv <= w.at) lo = mid;
            else hi = mid - 1;
        }
        w.b = lo;
    }
    // The stretch that begins at w.at: its unit, its blocks, and w.at moved behind it.
    auto open_stretch = [&](Walk& w, int ring) {
        while (sh.cost[w.b + 1] * Hkv <= w.at) ++w.b;
        w.len = p.t.len[w.b];
        w.n = blocks_of(w.len, w.lo);
        w.seen = window < 0 ? 0 : max(0, w.len - S_q - window);
        const unsigned into = w.at - sh.cost[w.b] * Hkv, per = paged_cost(w.n);
        w.h = (int)(into / per);
        const unsigned off = into - w.h * per, to = min(per, off + (w.end - w.at));
        w.g0 = min(w.n, max(0, (int)off - (int)kPagedOverhead));
        w.g1 = min(w.n, max(0, (int)to - (int)kPagedOverhead));
        w.g = w.g0 + ring;
        w.at += to - off;
    };

    const uint32_t ring_smem0 = smem_u32(ring_base);
    const uint32_t scale_smem0 = ring_smem0 + kRings * kStages * C::kBlockBytes;

    // =================================================== the loading warps: one for each ring
    if (warp >= kWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLoadRegs));
        const int ring = warp - kWarps;
        if (ring >= kRings) return;
        const uint32_t dst0 = ring_smem0 + ring * kStages * C::kBlockBytes;
        const uint32_t scale0 = scale_smem0 + ring * kStages * C::kScaleBytes;
        const uint32_t full0 = smem_u32(&sh.full[ring * kStages]), empty0 = smem_u32(&sh.empty[ring * kStages]);
        w.g = w.g1 = 0;
        // A batch: up to 32 blocks of the ring in one stretch, a lane each.  The next batch's page numbers are on their
        // way while this one's blocks are issued.
        struct Batch {
            int n;
            int unit[C::kBoxes], slot[C::kBoxes];  // page * Hkv + head, -1: the box is not needed
        };
        auto fetch = [&](Batch& f) {
            f.n = 0;
            while (w.g >= w.g1) {
                if (w.at >= w.end) return;
                open_stretch(w, ring);
            }
            f.n = min(32, (w.g1 - w.g + kRings - 1) / kRings);
            const int first = (w.lo + w.g + lane * kRings) * C::kKeys;
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
            w.g += 32 * kRings;
        };
        int fill = 0;
        uint32_t parity = 1;  // of the slot's last emptying; the first round finds every slot empty
        Batch now, then;
        fetch(now);
        while (now.n) {
            fetch(then);
            for (int i = 0; i < now.n; ++i) {
                bool stop = false;
                if (!mbar_try_wait(empty0 + 8 * fill, parity)) {
                    const uint64_t t0 = globaltimer();
                    while (!stop && !mbar_try_wait(empty0 + 8 * fill, parity))
                        stop = (long long)(globaltimer() - t0) > 2 * p.watchdog_ns;
                }
                // the computing warps have stopped (their own wait ran out and is recorded): stop as well
                if (__any_sync(0xFFFFFFFFu, stop)) return;
                const uint32_t bar = full0 + 8 * fill;
                int unit[C::kBoxes], slot[C::kBoxes], boxes = 0;
#pragma unroll
                for (int k = 0; k < C::kBoxes; ++k) {
                    unit[k] = __shfl_sync(0xFFFFFFFFu, now.unit[k], i);
                    slot[k] = __shfl_sync(0xFFFFFFFFu, now.slot[k], i);
                    boxes += unit[k] >= 0;
                }
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar, boxes * (C::kBoxBytes + (E4M3 ? 32 : 0)));
#pragma unroll
                    for (int k = 0; k < C::kBoxes; ++k) {
                        if (unit[k] < 0) continue;
                        tma_load_box(dst0 + fill * C::kBlockBytes + k * C::kBoxBytes, &p.tm, bar, slot[k], unit[k]);
                        if (E4M3)
                            bulk_load(scale0 + fill * C::kScaleBytes + 32 * k,
                                      p.c.scales + ((long long)unit[k] * (p.c.page / 16) + slot[k] / 16) * 32, 32, bar);
                    }
                }
                if (++fill == kStages) {
                    fill = 0;
                    parity ^= 1;
                }
            }
            now = then;
        }
        return;
    }

    // =================================================== the computing warps
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kComputeRegs));
    const int ring = warp / RW, rw = warp % RW;
    const int quad = lane / 4, pair = lane % 4;
    const uint32_t ring_smem = ring_smem0 + ring * kStages * C::kBlockBytes;
    const uint32_t scale_smem = scale_smem0 + ring * kStages * C::kScaleBytes;
    const uint32_t full = smem_u32(&sh.full[ring * kStages]), empty = smem_u32(&sh.empty[ring * kStages]);
    const float ninf = __int_as_float(0xFF800000);
    constexpr int kTiles = C::kKeys / 8;  // score tiles of a block
    bool dead = false;  // a wait ran out: nothing more is waited for, and the outputs are undefined
    int stage = 0;
    uint32_t phase = 0;
    while (w.at < w.end) {
        open_stretch(w, ring);
        if (w.g0 >= w.g1) continue;  // overhead alone (the same for every warp of the CTA)
        const int len = w.len, seen = w.seen;
        const int row0 = 16 * rw;
        // rows quad and quad + 8 of the warp's 16: their last and first visible position
        int last[2], first_seen[2];
        // The queries as the first operand.  bf16: qf[step][..] of 16 elements.  E4M3: a row is scaled by 2^-up to at
        // most 448 and split into two E4M3 numbers an element, qf[2 step] + 2^-4 qf[2 step + 1], 32 elements a step:
        // all eight bits of a bf16 number, down to 2^-22 of the row's largest.
        uint32_t qf[D / 16][4];
        float up[2] = {1.f, 1.f};  // 2^up of the rows
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
                if (E4M3) {
                    uint2 v[D / 16];
#pragma unroll
                    for (int i = 0; i < D / 16; ++i)
                        v[i] = real ? *reinterpret_cast<const uint2*>(qr + 16 * i + 4 * pair) : make_uint2(0, 0);
                    uint32_t big = 0;  // the largest magnitude, as bits of a bf16
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        big = __vmaxu2(big, v[i].x & 0x7FFF7FFFu);
                        big = __vmaxu2(big, v[i].y & 0x7FFF7FFFu);
                    }
                    big = max(big & 0xFFFFu, big >> 16);
                    big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, 1));
                    big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, 2));
                    // exponent field f: the row's numbers are below 2^(f - 126), so below 2^8 after the scaling.  A row
                    // below 2^-100 is taken as zeros; one with an infinity or a NaN becomes NaN.
                    const int f = (int)(big >> 7);
                    const float down = f == 255 ? __int_as_float(0x7FFFFFFF) : __uint_as_float((uint32_t)(261 - max(f, 27)) << 23);
                    up[r] = f == 255 ? __int_as_float(0x7FFFFFFF) : __uint_as_float((uint32_t)(max(f, 27) - 7) << 23);
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        uint32_t hi, lo;
                        split_e4m3(__uint_as_float(v[i].x << 16) * down, __uint_as_float(v[i].x & 0xFFFF0000u) * down,
                                   __uint_as_float(v[i].y << 16) * down, __uint_as_float(v[i].y & 0xFFFF0000u) * down,
                                   16.f, hi, lo);
                        qf[2 * (i / 2)][2 * (i % 2) + r] = hi;
                        qf[2 * (i / 2) + 1][2 * (i % 2) + r] = lo;
                    }
                } else {
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        qf[ks][r] = real ? *reinterpret_cast<const uint32_t*>(qr + 16 * ks + 2 * pair) : 0u;
                        qf[ks][2 + r] = real ? *reinterpret_cast<const uint32_t*>(qr + 16 * ks + 8 + 2 * pair) : 0u;
                    }
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

        for (; w.g < w.g1; w.g += kRings) {
            const int first = (w.lo + w.g) * C::kKeys;
            const uint32_t buf = ring_smem + stage * C::kBlockBytes;
            const uint32_t sc = scale_smem + stage * C::kScaleBytes;
            if (!dead && !mbar_try_wait(full + 8 * stage, phase)) {
                const uint64_t t0 = globaltimer();
                while (!mbar_try_wait(full + 8 * stage, phase)) {
                    if ((long long)(globaltimer() - t0) > p.watchdog_ns) {
                        dead = true;
                        atomicOr(p.c.err, kCacheErrWait);
                        break;
                    }
                }
            }
            __syncwarp();
            if (first + C::kKeys > len || first < seen) {
                // positions past the length or before the window may hold anything: weight zero times a NaN is a
                // NaN, so their values become zero (their scores are masked below)
#pragma unroll 1
                for (int key = 0; key < C::kKeys; ++key) {
                    if (first + key >= seen && first + key < len) continue;
                    const uint32_t v = buf + (key / 16) * C::kBoxBytes + C::kBoxBytes / 2 + (key % 16) * C::kInner;
                    if (lane < C::kRowBytes / 16) {
                        const uint32_t at = v + (lane / (C::kInner / 16)) * 16 * C::kInner + (lane % (C::kInner / 16)) * 16;
                        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0) : "memory");
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
            }
            // ---- S = Q K^T, in base 2
            float s[kTiles][4];
            if constexpr (E4M3) {
                const float f0 = p.scale_log2 * up[0], f1 = p.scale_log2 * up[1];
#pragma unroll
                for (int j0 = 0; j0 < kTiles; j0 += 2) {
                    float s2[2][4];
#pragma unroll
                    for (int k2 = 0; k2 < D / 64; ++k2) {
                        // one x4 load: 8 keys, 64 bytes of the row (two steps)
#pragma unroll
                        for (int jj = 0; jj < 2; ++jj) {
                            const int row = 8 * jj + lane % 8, chunk = 4 * k2 + lane / 8;
                            const int sw = C::kInner == 128 ? chunk ^ (row & 7) : chunk ^ ((row >> 1) & 3);
                            uint32_t r[4];
                            ldm4(r, buf + (j0 / 2) * C::kBoxBytes + row * C::kInner + sw * 16);
                            if (k2 == 0) {
                                mma_e4m3_first(s[j0 + jj], qf[0], r[0], r[1]);
                                mma_e4m3_first(s2[jj], qf[1], r[0], r[1]);
                            } else {
                                mma_e4m3(s[j0 + jj], qf[4 * k2], r[0], r[1]);
                                mma_e4m3(s2[jj], qf[4 * k2 + 1], r[0], r[1]);
                            }
                            mma_e4m3(s[j0 + jj], qf[4 * k2 + 2], r[2], r[3]);
                            mma_e4m3(s2[jj], qf[4 * k2 + 3], r[2], r[3]);
                        }
                    }
#pragma unroll
                    for (int jj = 0; jj < 2; ++jj) {
                        const int j = j0 + jj;
                        const uint32_t e = lds_u16(sc + 32 * (j / 2) + 8 * (j % 2) + 2 * pair);
                        const float k0 = exponent_factor(e & 255), k1 = exponent_factor(e >> 8);
                        s[j][0] = fmaf(s2[jj][0], 0.0625f, s[j][0]) * (k0 * f0);
                        s[j][1] = fmaf(s2[jj][1], 0.0625f, s[j][1]) * (k1 * f0);
                        s[j][2] = fmaf(s2[jj][2], 0.0625f, s[j][2]) * (k0 * f1);
                        s[j][3] = fmaf(s2[jj][3], 0.0625f, s[j][3]) * (k1 * f1);
                    }
                }
            } else {
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
                        ldm4(r, buf + bx * C::kBoxBytes + (ks / 4) * 16 * C::kInner + row * C::kInner +
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
            if constexpr (E4M3) {
                // Weights times the value rows' factors, x = s - m + k, brought to at most 2^8 for this block and row, as two
                // E4M3 numbers each (2^-8 of a weight, 2^-18 of the block's largest), against the codes themselves.
                float bx[2] = {ninf, ninf};
#pragma unroll
                for (int j = 0; j < kTiles; ++j) {
                    const uint32_t e = lds_u16(sc + 32 * (j / 2) + 16 + 8 * (j % 2) + 2 * pair);
                    // float(e - 127) through the significand of 2^23
                    const float v0 = __uint_as_float(0x4B000000u | (e & 255)) - 8388735.f;
                    const float v1 = __uint_as_float(0x4B000000u | (e >> 8)) - 8388735.f;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        // the reference first: what is left is small, and adding the exponent loses nothing
                        s[j][i] -= base[i >> 1];
                        l[i >> 1] += ex2(s[j][i]);
                        s[j][i] += i & 1 ? v1 : v0;
                    }
                    bx[0] = fmax3(bx[0], s[j][0], s[j][1]);
                    bx[1] = fmax3(bx[1], s[j][2], s[j][3]);
                }
                float back[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    bx[r] = fmaxf(bx[r], __shfl_xor_sync(0xFFFFFFFFu, bx[r], 1));
                    bx[r] = fmaxf(bx[r], __shfl_xor_sync(0xFFFFFFFFu, bx[r], 2));
                    const bool none = bx[r] == ninf;
                    bx[r] = none ? 0.f : bx[r] - 8.f;
                    back[r] = none ? 0.f : ex2(bx[r]);
                }
                uint32_t ph[4], pl[4];  // rows quad, quad + 8 of positions 0-15, then of 16-31
#pragma unroll
                for (int j = 0; j < kTiles; j += 2) {
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        float y[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) y[i] = ex2(s[j + i / 2][2 * r + i % 2] - bx[r]);
                        split_e4m3(y[0], y[1], y[2], y[3], 1.f, ph[j + r], pl[j + r]);
                    }
                }
                // one x4 load: 16 bytes of all 32 rows.  The transposing load hands out two bytes (an even and an odd
                // element) of two rows at a time; four rows of one element are put together from two of its registers.
                // The order of positions this gives, 2t, 2t + 1, 2t + 8, 2t + 9, is the order in ph and pl.
#pragma unroll
                for (int c = 0; c < D / 16; ++c) {
                    const int row = lane % 16;
                    const int sw = C::kInner == 128 ? c ^ (row & 7) : c ^ ((row >> 1) & 3);
                    uint32_t r[4];
                    ldm4t(r, buf + (lane / 16) * C::kBoxBytes + C::kBoxBytes / 2 + row * C::kInner + sw * 16);
                    const uint32_t e0 = __byte_perm(r[0], r[1], 0x6420), e1 = __byte_perm(r[2], r[3], 0x6420);
                    const uint32_t o0 = __byte_perm(r[0], r[1], 0x7531), o1 = __byte_perm(r[2], r[3], 0x7531);
                    float even[4], odd[4];
                    mma_e4m3_first(even, ph, e0, e1);
                    mma_e4m3_first(odd, ph, o0, o1);
                    mma_e4m3(even, pl, e0, e1);
                    mma_e4m3(odd, pl, o0, o1);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        acc[2 * c][i] = fmaf(even[i], back[i >> 1], acc[2 * c][i]);
                        acc[2 * c + 1][i] = fmaf(odd[i], back[i >> 1], acc[2 * c + 1][i]);
                    }
                }
            } else {
                uint32_t pf[C::kBoxes][4];
#pragma unroll
                for (int j = 0; j < kTiles; ++j) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        s[j][i] = ex2(s[j][i] - base[i >> 1]);
                        l[i >> 1] += s[j][i];
                    }
                    pf[j / 2][2 * (j % 2)] = pack_bf16x2(s[j][0], s[j][1]);
                    pf[j / 2][2 * (j % 2) + 1] = pack_bf16x2(s[j][2], s[j][3]);
                }
#pragma unroll
                for (int bx = 0; bx < C::kBoxes; ++bx) {
#pragma unroll
                    for (int c2 = 0; c2 < D / 16; ++c2) {
                        const int row = lane % 16, chunk = (2 * c2 + lane / 16) % 8;
                        uint32_t r[4];
                        ldm4t(r, buf + bx * C::kBoxBytes + C::kBoxBytes / 2 + (c2 / 4) * 16 * C::kInner + row * C::kInner +
                                     (chunk ^ (row & 7)) * 16);
                        mma_bf16(acc[2 * c2], pf[bx], r[0], r[1]);
                        mma_bf16(acc[2 * c2 + 1], pf[bx], r[2], r[3]);
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
                            const int col = E4M3 ? 16 * (jj / 2) + 4 * pair + 2 * i + jj % 2 : 8 * jj + 2 * pair + i;
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
        if (!final && w.g0 == 0 && tid == 0) {  // the unit begins here: where its last part is
            const unsigned u0 = sh.cost[w.b] * Hkv + w.h * paged_cost(w.n) + kPagedOverhead;
            p.cut[blockIdx.x] = make_int2(unit, (int)cuts.owner(u0 + w.n - 1));
        }
        named_bar_sync(1, 32 * kWarps);  // sh.ml and sh.red are free again
    }
    // after a wait that ran out, copies of this ring may still be on their way: wait for them, with a limit
    if (dead) {
        const uint64_t t0 = globaltimer();
        while (globaltimer() - t0 < 10000000ULL) __nanosleep(1000);
    }
}

// Joins the parts of the unit that begins in decode CTA blockIdx.x and ends in a later one: O = sum_k 2^(m_k - M) O_k / L
// with M = max m_k, L = sum_k 2^(m_k - M) l_k.  A warp per row.  The first part is in its CTA's second slot (the unit
// begins inside the interval), the others in their CTA's first.
constexpr int kMergeWarps = 8;
template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps) paged_merge_kernel(const __grid_constant__ PagedParams p, int rows_pad) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int row = blockIdx.y * kMergeWarps + threadIdx.x / 32, lane = threadIdx.x % 32;
    const int k0 = blockIdx.x;
    const int2 cut = __ldcg(&p.cut[k0]);
    if (cut.x < 0 || row >= p.rows) return;
    const int unit = cut.x, k1 = cut.y;
    const float ninf = __int_as_float(0xFF800000);
    auto at = [&](int k) { return (long long)(2 * k + (k == k0)) * rows_pad + row; };
    float M = ninf, L = 0.f;
    constexpr int kVec = D / 32;
    float v[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) v[i] = 0.f;
    for (int k = k0 + lane; k <= k1; k += 32) M = fmaxf(M, __ldcg(&p.part_ml[at(k)]).x);
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
    for (int kk = k0; kk <= k1; kk += 32) {
        float f = 0.f;
        if (kk + lane <= k1) {
            const float2 t = __ldcg(&p.part_ml[at(kk + lane)]);
            // a part without a maximum has seen nothing (sum 0), or only NaN
            f = t.x == ninf ? t.y : ex2(t.x - M);
            L += t.x == ninf ? t.y : t.y * f;
        }
        const int n = min(32, k1 - kk + 1);
#pragma unroll 8
        for (int i = 0; i < n; ++i) {
            const float fi = __shfl_sync(0xFFFFFFFFu, f, i);
            const float* src = p.part_o + at(kk + i) * D;
            if constexpr (D == 128) {
                const float4 y = __ldcg(reinterpret_cast<const float4*>(src) + lane);
                v[0] += fi * y.x; v[1] += fi * y.y; v[2] += fi * y.z; v[3] += fi * y.w;
            } else {
                const float2 y = __ldcg(reinterpret_cast<const float2*>(src) + lane);
                v[0] += fi * y.x; v[1] += fi * y.y;
            }
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xFFFFFFFFu, L, o);
    const float inv = L == 0.f ? 0.f : 1.f / L;
    uint32_t* o = reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(p.o) + ((long long)unit * p.rows + row) * D) +
                  lane * (D / 64);
#pragma unroll
    for (int i = 0; i < D / 64; ++i) o[i] = pack_bf16x2(v[2 * i] * inv, v[2 * i + 1] * inv);
    if (p.lse && lane == 0) p.lse[(long long)unit * p.rows + row] = (M + log2f(L)) * 0.6931471805599453f;
}

template <int D, bool E4M3, int RW>
cudaError_t launch_rw(const PagedParams& p, int grid, cudaStream_t stream) {
    const int smem = 1024 + Ring<D, E4M3, RW>::kBytes + (int)sizeof(Shared);
    static_assert(1024 + Ring<D, E4M3, RW>::kBytes + sizeof(Shared) <= 115712, "two CTAs per multiprocessor");
    auto* f = paged_kernel<D, E4M3, RW>;
    cudaError_t e = smem_opt_in(reinterpret_cast<const void*>(f), smem);
    if (e != cudaSuccess) return e;
    f<<<grid, kThreads, smem, stream>>>(p);
    return cudaGetLastError();
}
template <int D, bool E4M3>
cudaError_t launch_d(const PagedParams& p, int grid, cudaStream_t stream) {
    switch (paged_rows_pad(p.rows)) {
        case 16: return launch_rw<D, E4M3, 1>(p, grid, stream);
        case 32: return launch_rw<D, E4M3, 2>(p, grid, stream);
        default: return launch_rw<D, E4M3, 4>(p, grid, stream);
    }
}

}  // namespace

int paged_block_keys(int d, bool e4m3) {
    return d == 64 ? (e4m3 ? Cfg<64, true>::kKeys : Cfg<64, false>::kKeys)
                   : (e4m3 ? Cfg<128, true>::kKeys : Cfg<128, false>::kKeys);
}
int paged_rows_pad(int rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }
int paged_ctas_per_sm() { return kCtasPerSm; }

cudaError_t launch_paged_decode(const PagedParams& p, bool e4m3, int grid, bool merge, cudaStream_t stream) {
    cudaError_t e;
    if (p.c.d == 64) e = e4m3 ? launch_d<64, true>(p, grid, stream) : launch_d<64, false>(p, grid, stream);
    else e = e4m3 ? launch_d<128, true>(p, grid, stream) : launch_d<128, false>(p, grid, stream);
    if (e != cudaSuccess || !merge) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid, (unsigned)((p.rows + kMergeWarps - 1) / kMergeWarps));
    cfg.blockDim = dim3(32 * kMergeWarps);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const int pad = paged_rows_pad(p.rows);
    return p.c.d == 64 ? cudaLaunchKernelEx(&cfg, paged_merge_kernel<64>, p, pad)
                       : cudaLaunchKernelEx(&cfg, paged_merge_kernel<128>, p, pad);
}

}  // namespace attn
