// Attention of a few new rows per sequence over a paged cache (bf16 or E4M3).
//
//     O_i = sum_j softmax_j(scale q_i . k_j) v_j over the cached positions j that row i sees.
//
// Bound by memory: every visible key and value row is read once per kv head, for 4 * rows flops per element
// read, rows = the query rows that share the kv head (up to 64).
//
// A persistent grid, one CTA of eight warps per multiprocessor.  Lengths and page table are read on the device,
// so that a captured launch follows them: every CTA computes the same prefix sums of the lengths and takes an equal
// interval of the cost line (paged.h).  Inside a CTA the key blocks of a stretch (a CTA's part of a unit) go to the
// warps in turn.  Each warp, or each RW warps where there are more than 16 rows, has a ring of its own in shared
// memory, filled by one TMA box per 16 positions (keys and values of a head in one box, so that pages of any multiple of
// 16 work) and emptied without any barrier between the rings: a warp holds its own running maximum, sum and output
// tile (16 rows x d, fp32 registers) until the stretch ends.  Then the warps' results are added through shared
// memory, and a unit cut between CTAs is joined by the last of them to finish: partial results in slot order,
// so that the result does not depend on the order of arrival.
//
// The products are m16n8k16 bf16 with fp32 accumulation, rows padded to 16.  Their rate is not the limit: at the
// measured copy bandwidth an SM takes in about 24 bytes a clock, 12 bf16 elements, 188 multiply-adds at 16 rows.
// P is rounded to bf16 for the second product (relative 2^-9 a weight, below the rounding of O itself once summed);
// its row sum is taken before that rounding.  E4M3 codes become bf16 in registers, exactly: the seven low bits
// moved under the bf16 exponent are the value times 2^-120, one multiplication restores it.  A key row's factor 2^k
// multiplies its scores, a value row's its weights, both exact.
#include <cuda_bf16.h>

#include <algorithm>
#include <cstddef>

#include "device_once.h"
#include "paged.h"
#include "sm103_ptx.h"

namespace attn {

using namespace ptx;

namespace {

constexpr int kWarps = 8;
constexpr int kRedCols = 32;   // columns of the output added through shared memory at a time
constexpr int kRedPitch = 36;  // floats

template <int D, bool E4M3>
struct Cfg {
    static constexpr int kRowBytes = D * (E4M3 ? 1 : 2);
    static constexpr int kInner = kRowBytes < 128 ? kRowBytes : 128;  // bytes of a row part in shared memory
    static constexpr int kBoxBytes = 2 * 16 * kRowBytes;              // keys and values of 16 positions
    static constexpr int kBoxes = kBoxBytes >= 8192 ? 1 : 2;
    static constexpr int kKeys = 16 * kBoxes;                         // positions of a key block
    static constexpr int kBlockBytes = kBoxes * kBoxBytes;
    static constexpr int kScaleBytes = E4M3 ? 32 * kBoxes : 0;
    static constexpr int kTotal = 192 * 1024;                         // of all rings
    static_assert(kBoxBytes % 1024 == 0 && kScaleBytes % 16 == 0, "alignment of boxes and of what follows the rings");
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
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Four E4M3 codes to bf16: lo = codes 0 and 2, hi = codes 1 and 3.
__device__ __forceinline__ void e4m3_to_bf16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    const uint32_t l = ((w << 8) & 0x80008000u) | ((w << 4) & 0x07F007F0u);
    const uint32_t h = (w & 0x80008000u) | ((w >> 4) & 0x07F007F0u);
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(lo) : "r"(l), "r"(0x7B807B80u));
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(hi) : "r"(h), "r"(0x7B807B80u));
}
__device__ __forceinline__ float exponent_factor(int e) {  // 2^(e - 127); NaN for 255
    return __uint_as_float(e == 0 ? 0x00400000u : e == 255 ? 0x7FFFFFFFu : (uint32_t)e << 23);
}

// Where a warp stands in its CTA's interval of the cost line.
struct Walk {
    long long at, end;  // cost positions
    int b, h, n;        // current unit and its key blocks
    int g, g1;          // blocks [g, g1) of the stretch still to take (g advances by the number of rings)
    int g0;             // first block of the stretch
    int lo;             // first key block of the sequence
    int len, seen;      // its visible positions: [seen, len)
};

// Shared memory of a CTA besides the rings (behind them).
struct Shared {
    long long cost[kPagedMaxBatch + 1];  // cost of the sequences before b
    alignas(16) float red[kWarps * 16 * kRedPitch];  // read as float4
    float2 ml[kWarps * 16];
    float2 row[64];                      // maximum and sum of the rows of the stretch
    unsigned long long bars[kWarps * 8];
    long long scan[kWarps];
    int last;
};
static_assert(offsetof(Shared, red) % 16 == 0 && offsetof(Shared, bars) % 8 == 0 && offsetof(Shared, ml) % 8 == 0 &&
                  alignof(Shared) == 16 && kRedPitch % 4 == 0,
              "alignment of the shared accesses");

template <int D, bool E4M3, int RW>
__global__ void __launch_bounds__(kWarps * 32, 1) paged_kernel(const __grid_constant__ PagedParams p) {
    using C = Cfg<D, E4M3>;
    constexpr int kRings = kWarps / RW;
    constexpr int kStages = C::kTotal / kRings / C::kBlockBytes < 6 ? C::kTotal / kRings / C::kBlockBytes : 6;
    constexpr int kSteps = D / 16;
    extern __shared__ uint8_t smem_raw[];
    // boxes are swizzled by address: the rings begin on a 1024-byte boundary
    uint8_t* const ring_base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    Shared& sh = *reinterpret_cast<Shared*>(ring_base + kRings * kStages * (C::kBlockBytes + C::kScaleBytes));
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int ring = warp / RW, rw = warp % RW;
    const int quad = lane / 4, pair = lane % 4;
    const int Hkv = p.Hkv, S_q = p.S_q, window = p.window;

    // ---- prefix sums of the sequences' cost
    const int room = (int)min((long long)p.t.max_pages * p.c.page, 0x7FFFFF00LL);
    auto blocks_of = [&](int b, int& lo) {
        int n = p.t.len[b];
        if (n < 0 || n > room) n = 0;
        int hi;
        paged_blocks(n, S_q, window, C::kKeys, lo, hi);
        return hi - lo;
    };
    if (tid < kRings * kStages) mbar_init(smem_u32(&sh.bars[tid]), 1);
    if (tid == 0) {
        prefetch_tmap(&p.tm);
        sh.cost[0] = 0;
    }
    long long carry = 0;
    int busy = 0;  // sequences with keys
    for (int b0 = 0; b0 < p.B; b0 += kWarps * 32) {
        const int b = b0 + tid;
        long long x = 0, cost = 0;
        if (b < p.B) {
            int lo;
            const int n = blocks_of(b, lo);
            x = cost = n ? (long long)Hkv * (n + kPagedOverhead) : 0;
            const int len = p.t.len[b];
            if (blockIdx.x == 0 && (len < 0 || len > room)) atomicOr(p.c.err, kCacheErrPosition);
        }
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const long long y = __shfl_up_sync(0xFFFFFFFFu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) sh.scan[warp] = x;
        busy += __syncthreads_count(b < p.B && cost != 0);
        long long before = carry, all = carry;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) before += sh.scan[w];
            all += sh.scan[w];
        }
        if (b < p.B) sh.cost[b + 1] = before + x;
        carry = all;
        __syncthreads();
    }
    fence_barrier_init();
    __syncthreads();
    const long long W = carry;
    const int n_cta = paged_ctas(W, busy * Hkv, gridDim.x, kRings + kPagedOverhead);

    // ---- sequences without keys: rows of zeros, LSE -inf
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        if (sh.cost[b + 1] != sh.cost[b]) continue;
        uint4* o = reinterpret_cast<uint4*>(p.o) + (long long)b * p.Hq * S_q * (D / 8);
        for (int i = tid; i < p.Hq * S_q * (D / 8); i += kWarps * 32) o[i] = make_uint4(0, 0, 0, 0);
        if (p.lse)
            for (int i = tid; i < p.Hq * S_q; i += kWarps * 32)
                p.lse[(long long)b * p.Hq * S_q + i] = __int_as_float(0xFF800000);
    }
    if ((int)blockIdx.x >= n_cta || W == 0) return;

    // ---- the CTA's interval
    Walk start;
    start.at = paged_cut(W, n_cta, blockIdx.x);
    start.end = paged_cut(W, n_cta, blockIdx.x + 1);
    {
        int lo = 0, hi = p.B - 1;  // the last b with cost[b] <= at (and cost[b + 1] > at)
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (sh.cost[mid] <= start.at) lo = mid;
            else hi = mid - 1;
        }
        start.b = lo;
    }
    // The stretch that begins at w.at: its unit, its blocks, and w.at moved behind it.
    auto open_stretch = [&](Walk& w) {
        while (sh.cost[w.b + 1] <= w.at) ++w.b;
        w.n = blocks_of(w.b, w.lo);
        w.len = p.t.len[w.b];
        w.seen = window < 0 ? 0 : max(0, w.len - S_q - window);
        const long long into = w.at - sh.cost[w.b];
        const int per = w.n + kPagedOverhead;
        w.h = (int)(into / per);
        const int off = (int)(into - (long long)w.h * per);
        const long long to = min((long long)per, off + (w.end - w.at));
        w.g0 = max(0, off - kPagedOverhead);
        w.g1 = max(0, (int)to - kPagedOverhead);
        w.g = w.g0 + ring;
        w.at += to - off;
    };

    const uint32_t ring_smem = smem_u32(ring_base) + ring * kStages * C::kBlockBytes;
    const uint32_t scale_smem = smem_u32(ring_base) + kRings * kStages * C::kBlockBytes + ring * kStages * C::kScaleBytes;
    const uint32_t bars = smem_u32(&sh.bars[ring * kStages]);

    // ---- the loading side (warp rw = 0 of a ring): its own walk, kStages blocks ahead
    Walk in = start;
    in.g = in.g1 = 0;
    int fill = 0;
    bool dead = false;  // a wait ran out: nothing more is loaded or waited for, and the outputs are undefined
    auto issue = [&]() {
        while (in.g >= in.g1) {
            if (in.at >= in.end) return;
            open_stretch(in);
        }
        const int first = (in.lo + in.g) * C::kKeys;
        const uint32_t dst = ring_smem + fill * C::kBlockBytes, bar = bars + 8 * fill;
        int box_page = 0, box_slot = 0;
        bool have = false;
        if (lane < C::kBoxes) {  // lane k takes the 16 positions from first + 16 k
            const int pos = first + 16 * lane;
            have = pos < in.len && pos + 16 > in.seen;
            if (have) {
                const int index = pos / p.c.page;
                box_slot = pos - index * p.c.page;
                box_page = p.t.pages[in.b * p.t.stride + index];
                if (box_page < 0 || box_page >= p.c.n_pages) {
                    atomicOr(p.c.err, kCacheErrPage);
                    box_page = 0;
                }
            }
        }
        const int boxes = __popc(__ballot_sync(0xFFFFFFFFu, have));
        if (lane == 0) mbar_arrive_expect_tx(bar, boxes * (C::kBoxBytes + (E4M3 ? 32 : 0)));
        __syncwarp();
        if (have) {
            const int unit = box_page * Hkv + in.h;
            tma_load_box(dst + lane * C::kBoxBytes, &p.tm, bar, box_slot, unit);
            if (E4M3)
                bulk_load(scale_smem + fill * C::kScaleBytes + 32 * lane,
                          p.c.scales + ((long long)unit * (p.c.page / 16) + box_slot / 16) * 32, 32, bar);
        }
        fill = fill + 1 == kStages ? 0 : fill + 1;
        in.g += kRings;
    };
    if (rw == 0)
        for (int s = 0; s < kStages; ++s) issue();

    // ---- the computing side
    Walk w = start;
    int stage = 0;
    uint32_t phase = 0;
    while (w.at < w.end) {
        open_stretch(w);
        if (w.g0 >= w.g1) continue;  // overhead alone (the same for every warp of the CTA)
        const int len = w.len, seen = w.seen;
        const int row0 = 16 * rw;
        // rows quad and quad + 8 of the warp's 16: their last and first visible position
        int last[2], first_seen[2];
        uint32_t qf[kSteps][4];
        {
            const __nv_bfloat16* q =
                reinterpret_cast<const __nv_bfloat16*>(p.q) + ((long long)w.b * Hkv + w.h) * p.rows * D;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = row0 + quad + 8 * r;
                const bool real = row < p.rows;
                const int t = len - S_q + row % S_q;
                last[r] = !real ? -1 : p.causal ? t : len - 1;
                first_seen[r] = window < 0 ? 0 : max(0, t - window);
                const uint16_t* qr = reinterpret_cast<const uint16_t*>(q + (long long)row * D);
#pragma unroll
                for (int ks = 0; ks < kSteps; ++ks) {
                    uint32_t a = 0, b = 0;
                    if (real) {
                        if (E4M3) {  // the order e4m3_to_bf16 leaves the keys' elements in
                            const uint2 v = *reinterpret_cast<const uint2*>(qr + 16 * ks + 4 * pair);
                            a = __byte_perm(v.x, v.y, 0x5410);
                            b = __byte_perm(v.x, v.y, 0x7632);
                        } else {
                            a = *reinterpret_cast<const uint32_t*>(qr + 16 * ks + 2 * pair);
                            b = *reinterpret_cast<const uint32_t*>(qr + 16 * ks + 8 + 2 * pair);
                        }
                    }
                    qf[ks][r] = a;
                    qf[ks][2 + r] = b;
                }
            }
        }
        // positions every real row sees need no test: [all_from, all_to)
        const int all_to = p.causal ? len - S_q + 1 : len;
        const int all_from = window < 0 ? 0 : len - 1 - window;
        float acc[D / 8][4];
#pragma unroll
        for (int j = 0; j < D / 8; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
        const float ninf = __int_as_float(0xFF800000);
        float m[2] = {ninf, ninf}, l[2] = {0.f, 0.f};

        for (; w.g < w.g1; w.g += kRings) {
            const int first = (w.lo + w.g) * C::kKeys;
            const uint32_t buf = ring_smem + stage * C::kBlockBytes;
            const uint32_t sc = scale_smem + stage * C::kScaleBytes;
            if (!dead && !mbar_try_wait(bars + 8 * stage, phase)) {
                const uint64_t t0 = globaltimer();
                while (!mbar_try_wait(bars + 8 * stage, phase)) {
                    if ((long long)(globaltimer() - t0) > p.watchdog_ns) {
                        dead = true;
                        break;
                    }
                }
            }
            if (__any_sync(0xFFFFFFFFu, dead) && !dead) dead = true;
            if (dead && lane == 0) atomicOr(p.c.err, kCacheErrWait);
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
            float s[C::kKeys / 8][4];
#pragma unroll
            for (int j = 0; j < C::kKeys / 8; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
            // S = Q K^T
#pragma unroll
            for (int bx = 0; bx < C::kBoxes; ++bx) {
                const uint32_t kb = buf + bx * C::kBoxBytes;
                if (E4M3) {
                    // one x4 load: keys 0-7 and 8-15, 32 bytes of the row (two steps)
#pragma unroll
                    for (int k2 = 0; k2 < D / 32; ++k2) {
                        const int row = lane % 8 + 8 * ((lane / 8) & 1), chunk = 2 * k2 + lane / 16;
                        const int sw = C::kInner == 128 ? chunk ^ (row & 7) : chunk ^ ((row >> 1) & 3);
                        uint32_t r[4];
                        ldm4(r, kb + row * C::kInner + sw * 16);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            uint32_t b0, b1;
                            e4m3_to_bf16(r[q], b0, b1);
                            const int ks = 2 * k2 + q / 2, nt = 2 * bx + q % 2;
                            mma16816(s[nt], qf[ks][0], qf[ks][1], qf[ks][2], qf[ks][3], b0, b1);
                        }
                    }
                } else {
                    // one x4 load: keys 0-7 and 8-15, 16 elements of the row (one step)
#pragma unroll
                    for (int ks = 0; ks < kSteps; ++ks) {
                        const int row = lane % 8 + 8 * (lane / 16), chunk = (2 * ks + (lane / 8 & 1)) % 8;
                        uint32_t r[4];
                        ldm4(r, kb + (ks / 4) * 16 * C::kInner + row * C::kInner + (chunk ^ (row & 7)) * 16);
                        mma16816(s[2 * bx], qf[ks][0], qf[ks][1], qf[ks][2], qf[ks][3], r[0], r[1]);
                        mma16816(s[2 * bx + 1], qf[ks][0], qf[ks][1], qf[ks][2], qf[ks][3], r[2], r[3]);
                    }
                }
            }
            // scores in base 2, masked; the block's row maxima
            const bool whole = first >= all_from && first + C::kKeys <= all_to;
            float top[2] = {ninf, ninf};
#pragma unroll
            for (int j = 0; j < C::kKeys / 8; ++j) {
                float f[2] = {p.scale_log2, p.scale_log2};
                if (E4M3) {
                    uint16_t e;
                    asm volatile("ld.shared.u16 %0, [%1];"
                                 : "=h"(e)
                                 : "r"(sc + 32 * (j / 2) + 8 * (j % 2) + 2 * pair)
                                 : "memory");
                    f[0] *= exponent_factor(e & 255);
                    f[1] *= exponent_factor(e >> 8);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float v = s[j][i] * f[i & 1];
                    if (!whole) {
                        const int pos = first + 8 * j + 2 * pair + (i & 1);
                        if (pos > last[i >> 1] || pos < first_seen[i >> 1]) v = ninf;
                    }
                    s[j][i] = v;
                    top[i >> 1] = fmaxf(top[i >> 1], v);
                }
            }
            // the maximum moves only when it is passed by 2^8: weights stay below 256, and the output is
            // rescaled rarely
            bool moved = false;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                top[r] = fmaxf(top[r], __shfl_xor_sync(0xFFFFFFFFu, top[r], 1));
                top[r] = fmaxf(top[r], __shfl_xor_sync(0xFFFFFFFFu, top[r], 2));
                moved |= top[r] > m[r] + 8.f;
            }
            if (__any_sync(0xFFFFFFFFu, moved)) {
                float fix[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float to = top[r] > m[r] + 8.f ? top[r] : m[r];
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
            uint32_t pf[C::kKeys / 8][2];
#pragma unroll
            for (int j = 0; j < C::kKeys / 8; ++j) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s[j][i] = ex2(s[j][i] - base[i >> 1]);
                    l[i >> 1] += s[j][i];
                }
                if (E4M3) {
                    uint16_t e;
                    asm volatile("ld.shared.u16 %0, [%1];"
                                 : "=h"(e)
                                 : "r"(sc + 32 * (j / 2) + 16 + 8 * (j % 2) + 2 * pair)
                                 : "memory");
                    // a masked position's factor may be anything
                    const int pos = first + 8 * j + 2 * pair;
                    const float f0 = pos >= seen && pos < len ? exponent_factor(e & 255) : 0.f;
                    const float f1 = pos + 1 >= seen && pos + 1 < len ? exponent_factor(e >> 8) : 0.f;
                    s[j][0] *= f0; s[j][2] *= f0;
                    s[j][1] *= f1; s[j][3] *= f1;
                }
                pf[j][0] = pack_bf16x2(s[j][0], s[j][1]);
                pf[j][1] = pack_bf16x2(s[j][2], s[j][3]);
            }
            // O += P V
#pragma unroll
            for (int bx = 0; bx < C::kBoxes; ++bx) {
                const uint32_t vb = buf + bx * C::kBoxBytes + C::kBoxBytes / 2;
                const uint32_t a0 = pf[2 * bx][0], a1 = pf[2 * bx][1], a2 = pf[2 * bx + 1][0], a3 = pf[2 * bx + 1][1];
                if (E4M3) {
                    // one x4 load: keys 0-7 and 8-15, 32 bytes: even and odd elements come apart as two tiles
#pragma unroll
                    for (int c2 = 0; c2 < D / 32; ++c2) {
                        const int row = lane % 8 + 8 * ((lane / 8) & 1), chunk = 2 * c2 + lane / 16;
                        const int sw = C::kInner == 128 ? chunk ^ (row & 7) : chunk ^ ((row >> 1) & 3);
                        uint32_t r[4];
                        ldm4t(r, vb + row * C::kInner + sw * 16);
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            uint32_t e0, e1, o0, o1;
                            e4m3_to_bf16(r[2 * c], e0, o0);
                            e4m3_to_bf16(r[2 * c + 1], e1, o1);
                            mma16816(acc[4 * c2 + 2 * c], a0, a1, a2, a3, e0, e1);
                            mma16816(acc[4 * c2 + 2 * c + 1], a0, a1, a2, a3, o0, o1);
                        }
                    }
                } else {
#pragma unroll
                    for (int c2 = 0; c2 < D / 16; ++c2) {
                        const int row = lane % 16, chunk = (2 * c2 + lane / 16) % 8;
                        uint32_t r[4];
                        ldm4t(r, vb + (c2 / 4) * 16 * C::kInner + row * C::kInner + (chunk ^ (row & 7)) * 16);
                        mma16816(acc[2 * c2], a0, a1, a2, a3, r[0], r[1]);
                        mma16816(acc[2 * c2 + 1], a0, a1, a2, a3, r[2], r[3]);
                    }
                }
            }
            stage = stage + 1 == kStages ? 0 : stage + 1;
            if (stage == 0) phase ^= 1;
            // the block is read: the next one into its place
            if (RW == 1) __syncwarp();
            else named_bar_sync(1 + ring, 32 * RW);
            if (rw == 0 && !dead) issue();
        }

        // ---- the warps' results of this stretch, added
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 1);
            l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 2);
            if (pair == 0) sh.ml[warp * 16 + quad + 8 * r] = make_float2(m[r], l[r]);
        }
        __syncthreads();
        if (tid < 16 * RW) {  // row tid of the unit
            float M = ninf, L = 0.f;
            for (int g = 0; g < kRings; ++g) M = fmaxf(M, sh.ml[(g * RW + tid / 16) * 16 + tid % 16].x);
            for (int g = 0; g < kRings; ++g) {
                const float2 v = sh.ml[(g * RW + tid / 16) * 16 + tid % 16];
                L += v.x == ninf ? v.y : v.y * ex2(v.x - M);
            }
            sh.row[tid] = make_float2(M, L);
        }
        __syncthreads();
        float fix[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) fix[r] = m[r] == ninf ? 0.f : ex2(m[r] - sh.row[row0 + quad + 8 * r].x);
        const bool final = w.g0 == 0 && w.g1 == w.n;
        const int unit = w.b * Hkv + w.h;
        const int slot = 2 * blockIdx.x + (w.g0 > 0 ? 0 : 1);
        constexpr int kRowsPad = 16 * RW;
        float* part = p.part_o + (long long)slot * kRowsPad * D;
#pragma unroll
        for (int c0 = 0; c0 < D; c0 += kRedCols) {
            // columns c0 .. c0 + 31 are the tiles c0 / 8 .. + 3
            float* mine = sh.red + warp * 16 * kRedPitch;
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int jj = 0; jj < 4; ++jj)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int col = E4M3 ? 16 * (jj / 2) + 4 * pair + 2 * i + jj % 2 : 8 * jj + 2 * pair + i;
                        mine[(quad + 8 * r) * kRedPitch + col] = acc[c0 / 8 + jj][2 * r + i] * fix[r];
                    }
            __syncthreads();
#pragma unroll
            for (int x = tid; x < kRowsPad * kRedCols / 4; x += kWarps * 32) {
                const int row = x / (kRedCols / 4), c4 = x % (kRedCols / 4) * 4;
                if (row >= p.rows) continue;
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int g = 0; g < kRings; ++g) {
                    const float4 y = *reinterpret_cast<const float4*>(
                        &sh.red[((g * RW + row / 16) * 16 + row % 16) * kRedPitch + c4]);
                    v.x += y.x; v.y += y.y; v.z += y.z; v.w += y.w;
                }
                if (final) {
                    const float L = sh.row[row].y;
                    const float inv = L == 0.f ? 0.f : 1.f / L;
                    uint2 o = make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
                    *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p.o) +
                                              ((long long)unit * p.rows + row) * D + c0 + c4) = o;
                } else {
                    __stcg(reinterpret_cast<float4*>(part + row * D + c0 + c4), v);
                }
            }
            __syncthreads();
        }
        if (tid < p.rows) {
            const float2 v = sh.row[tid];
            if (!final) __stcg(&p.part_ml[slot * kRowsPad + tid], v);
            else if (p.lse) p.lse[(long long)unit * p.rows + tid] = (v.x + log2f(v.y)) * 0.6931471805599453f;
        }
        if (!final) {
            // the CTAs that hold blocks of this unit; the last to arrive joins their results
            const int per = w.n + kPagedOverhead;
            const long long u0 = sh.cost[w.b] + (long long)w.h * per + kPagedOverhead;
            const int k0 = paged_owner(W, n_cta, u0), k1 = paged_owner(W, n_cta, u0 + w.n - 1);
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                const unsigned before = atomicAdd(&p.counters[unit], 1u);
                sh.last = before == (unsigned)(k1 - k0);
                if (sh.last) p.counters[unit] = 0;
            }
            __syncthreads();
            if (sh.last) {
                __threadfence();
                // a warp per row; the first CTA's slot is its second one (the unit begins inside its interval)
                for (int row = warp; row < p.rows; row += kWarps) {
                    float M = ninf;
                    for (int k = k0 + lane; k <= k1; k += 32)
                        M = fmaxf(M, __ldcg(&p.part_ml[(2 * k + (k == k0)) * kRowsPad + row]).x);
#pragma unroll
                    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
                    float L = 0.f;
                    float v[D / 32];
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) v[i] = 0.f;
                    for (int kk = k0; kk <= k1; kk += 32) {
                        const int mine_k = kk + lane;
                        float f = 0.f;
                        if (mine_k <= k1) {
                            const float2 t = __ldcg(&p.part_ml[(2 * mine_k + (mine_k == k0)) * kRowsPad + row]);
                            f = t.x == ninf ? (t.y == 0.f ? 0.f : t.y) : ex2(t.x - M);
                            L += t.x == ninf ? t.y : t.y * f;
                        }
                        const int n = min(32, k1 - kk + 1);
#pragma unroll 8
                        for (int i = 0; i < n; ++i) {
                            const int k = kk + i;
                            const float fi = __shfl_sync(0xFFFFFFFFu, f, i);
                            const float* src = p.part_o + ((long long)(2 * k + (k == k0)) * kRowsPad + row) * D;
                            if (D == 128) {
                                const float4 y = __ldcg(reinterpret_cast<const float4*>(src) + lane);
                                v[0] += fi * y.x; v[1] += fi * y.y; v[D / 32 - 2] += fi * y.z; v[D / 32 - 1] += fi * y.w;
                            } else {
                                const float2 y = __ldcg(reinterpret_cast<const float2*>(src) + lane);
                                v[0] += fi * y.x; v[1] += fi * y.y;
                            }
                        }
                    }
#pragma unroll
                    for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xFFFFFFFFu, L, o);
                    const float inv = L == 0.f ? 0.f : 1.f / L;
                    uint32_t* o = reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(p.o) +
                                                              ((long long)unit * p.rows + row) * D) + lane * (D / 64);
#pragma unroll
                    for (int i = 0; i < D / 64; ++i) o[i] = pack_bf16x2(v[2 * i] * inv, v[2 * i + 1] * inv);
                    if (p.lse && lane == 0)
                        p.lse[(long long)unit * p.rows + row] = (M + log2f(L)) * 0.6931471805599453f;
                }
            }
        }
    }
    // after a wait that ran out, copies of this ring may still be on their way: wait for them, with a limit
    if (dead) {
        const uint64_t t0 = globaltimer();
        while (globaltimer() - t0 < 10000000ULL) __nanosleep(1000);
    }
}

template <int D, bool E4M3, int RW>
cudaError_t launch_rw(const PagedParams& p, int grid, cudaStream_t stream) {
    using C = Cfg<D, E4M3>;
    constexpr int kRings = kWarps / RW;
    constexpr int kStages = C::kTotal / kRings / C::kBlockBytes < 6 ? C::kTotal / kRings / C::kBlockBytes : 6;
    const int smem = 1024 + kRings * kStages * (C::kBlockBytes + C::kScaleBytes) + (int)sizeof(Shared);
    auto* f = paged_kernel<D, E4M3, RW>;
    cudaError_t e = smem_opt_in(reinterpret_cast<const void*>(f), smem);
    if (e != cudaSuccess) return e;
    f<<<grid, kWarps * 32, smem, stream>>>(p);
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

cudaError_t launch_paged_decode(const PagedParams& p, bool e4m3, int grid, cudaStream_t stream) {
    if (p.c.d == 64) return e4m3 ? launch_d<64, true>(p, grid, stream) : launch_d<64, false>(p, grid, stream);
    return e4m3 ? launch_d<128, true>(p, grid, stream) : launch_d<128, false>(p, grid, stream);
}

}  // namespace attn
