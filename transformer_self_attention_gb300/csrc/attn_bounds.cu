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
// Select: a cluster of one to eight blocks for each sequence and kv head, four lanes to a page (each takes a quarter of the
// channels: 16 channels an instruction would need four dp4a of a product, which the scores' 2 d bytes a page are worth).
// Scores go to the first block's shared memory, which then finds the largest (select.h).
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

__device__ __forceinline__ float min_nan(float a, float b) {
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
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
template <>
struct RowBounds<true> {
    static constexpr int kChannels = 16;
    float lo[16], hi[16];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            lo[i] = __uint_as_float(0x7F800000u);
            hi[i] = __uint_as_float(0xFF800000u);
        }
    }
    __device__ __forceinline__ void take(const uint4& v, uint32_t e) {
        // 2^(e - 127), or NaN for 255
        const float f = e == 255 ? __uint_as_float(0x7FFFFFFFu) : __uint_as_float(max(e << 23, 0x00400000u));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t h2;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)(w[i / 2] >> 16 * (i % 2))));
            float a, b;
            asm("{.reg .f16 x, y; mov.b32 {x, y}, %2; cvt.f32.f16 %0, x; cvt.f32.f16 %1, y;}" : "=f"(a), "=f"(b) : "r"(h2));
            a *= f;
            b *= f;
            lo[2 * i] = min_nan(lo[2 * i], a);
            hi[2 * i] = max_nan(hi[2 * i], a);
            lo[2 * i + 1] = min_nan(lo[2 * i + 1], b);
            hi[2 * i + 1] = max_nan(hi[2 * i + 1], b);
        }
    }
    __device__ __forceinline__ void join(int o) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            lo[i] = min_nan(lo[i], __shfl_xor_sync(0xFFFFFFFFu, lo[i], o));
            hi[i] = max_nan(hi[i], __shfl_xor_sync(0xFFFFFFFFu, hi[i], o));
        }
    }
    __device__ __forceinline__ void get(float* l, float* h) const {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            l[i] = lo[i];
            h[i] = hi[i];
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

template <int D>
struct SelectMemory {
    alignas(16) int8_t q[ATTN_DECODE_MAX_ROWS][2][D];  // negative and positive parts
    SelectShared<kSelectThreads> sel;
    unsigned big[kSelectThreads / 32];
};

template <int D>
__global__ void __launch_bounds__(kSelectThreads) select_kernel(const __grid_constant__ SelectParams p) {
    __shared__ SelectMemory<D> sh;
    extern __shared__ uint32_t keys[];  // of the first block of the cluster: a page each
    const cg::cluster_group cluster = cg::this_cluster();
    const int blocks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int unit = blockIdx.x / blocks, b = unit / p.Hkv, h = unit - b * p.Hkv, page = p.c.page;
    wait_for_kernel_before();
    let_kernel_behind_in();
    const int len = sequence_length(p.t, page, b, p.c.err, tid == 0 && h == 0 && rank == 0);
    const int n = (unsigned)(len + page - 1) / (unsigned)page;
    const int* row = p.t.pages + b * p.t.stride;
    int* out = p.out_table + (long long)unit * p.keep;
    if (h == 0 && rank == 0 && tid == 0) p.out_len[b] = n > p.keep ? len - (n - p.keep) * page : len;
    if (n <= p.keep) {  // (the whole cluster)
        if (rank == 0)
            for (int i = tid; i < p.keep; i += kSelectThreads) out[i] = i < n ? row[i] : -1;
        return;
    }
    const int lo = p.sinks, m = n - p.recent - lo, K = p.keep - p.recent - lo;  // m > K >= 0
    if (rank == 0) {
        for (int i = tid; i < lo; i += kSelectThreads) out[i] = row[i];
        for (int i = tid; i < p.recent; i += kSelectThreads) out[lo + K + i] = row[n - p.recent + i];
    }
    if (K == 0) return;
    // the queries as whole numbers of one power of two
    const uint4* q = reinterpret_cast<const uint4*>(p.q) + (long long)unit * p.rows * (D / 8);
    uint32_t big = 0;  // as bits of a bf16
    for (int i = tid; i < p.rows * (D / 8); i += kSelectThreads) {
        const uint4 v = q[i];
        uint32_t t = __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
        big = max(big, max(t & 0xFFFFu, t >> 16));
    }
    big = __reduce_max_sync(0xFFFFFFFFu, big);
    if (lane == 0) sh.big[warp] = big;
    __syncthreads();
    big = __reduce_max_sync(0xFFFFFFFFu, sh.big[lane % (kSelectThreads / 32)]);
    const bool bad = big >= 0x7F80u;  // queries that are not finite choose the first pages
    const float f = bad ? 0.f : exp2_of(-power_of(big << 16));
    for (int i = tid; i < p.rows * (D / 8); i += kSelectThreads) {
        const uint4 v = q[i];
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t neg[2] = {0, 0}, pos[2] = {0, 0};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float x = __uint_as_float(j % 2 ? w[j / 2] & 0xFFFF0000u : w[j / 2] << 16);
            const int c = bad ? 0 : __float2int_rn(x * f);
            neg[j / 4] |= (uint32_t)(min(c, 0) & 0xFF) << 8 * (j % 4);
            pos[j / 4] |= (uint32_t)max(c, 0) << 8 * (j % 4);
        }
        const int r = i / (D / 8), c = i % (D / 8);
        *reinterpret_cast<uint2*>(&sh.q[r][0][8 * c]) = make_uint2(neg[0], neg[1]);
        *reinterpret_cast<uint2*>(&sh.q[r][1][8 * c]) = make_uint2(pos[0], pos[1]);
    }
    if (blocks > 1) cluster.sync();  // (all blocks of the cluster are there)
    else __syncthreads();
    uint32_t* first_keys = blocks > 1 ? cluster.map_shared_rank(keys, 0) : keys;
    constexpr int kPages = kSelectThreads / 4, kChunks = D / 64;  // 16-byte chunks of a lane and row
    const int quarter = lane % 4;
    for (int i0 = rank * kPages; i0 < m; i0 += blocks * kPages) {
        const int i = i0 + tid / 4;
        uint32_t c[2][4 * kChunks];
        int e = 0;
        if (i < m) {
            const int g = row[lo + i];
            const bool ok = g >= 0 && g < p.c.n_pages;
            if (!ok && h == 0 && quarter == 0) atomicOr(p.c.err, kCacheErrPage);
            const long long at = (long long)(ok ? g : 0) * p.Hkv + h;
            const uint4* src = reinterpret_cast<const uint4*>(p.codes + at * 2 * D);
            e = p.exps[at];
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int j = 0; j < kChunks; ++j) {
                    const uint4 v = src[s * (D / 16) + 4 * j + quarter];
                    c[s][4 * j] = v.x; c[s][4 * j + 1] = v.y; c[s][4 * j + 2] = v.z; c[s][4 * j + 3] = v.w;
                }
        } else {
#pragma unroll
            for (int j = 0; j < 4 * kChunks; ++j) c[0][j] = c[1][j] = 0;
        }
        int best = -(1 << 30);
        for (int r = 0; r < p.rows; ++r) {
            int sum = 0;
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int j = 0; j < kChunks; ++j) {
                    const uint4 v = *reinterpret_cast<const uint4*>(&sh.q[r][s][16 * (4 * j + quarter)]);
                    sum = __dp4a((int)v.x, (int)c[s][4 * j], sum);
                    sum = __dp4a((int)v.y, (int)c[s][4 * j + 1], sum);
                    sum = __dp4a((int)v.z, (int)c[s][4 * j + 2], sum);
                    sum = __dp4a((int)v.w, (int)c[s][4 * j + 3], sum);
                }
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
            best = max(best, sum);
        }
        if (i < m && quarter == 0)
            first_keys[i] = e == 255 ? 0xFF800000u : ordered((float)best * __uint_as_float((uint32_t)e << 23));
    }
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
    const int grid = (int)std::min<long long>((items + warps - 1) / warps, 4LL * n_sm);
    auto go = [&](auto* f) { return launch_dependent(f, dim3((unsigned)grid), kUpdateThreads, 0, stream, p); };
    if (p.c.d == 64) return e4m3 ? go(update_kernel<64, true>) : go(update_kernel<64, false>);
    return e4m3 ? go(update_kernel<128, true>) : go(update_kernel<128, false>);
}

cudaError_t launch_bounds_select(const SelectParams& p, int n_sm, cudaStream_t stream) {
    const int units = p.B * p.Hkv;
    int cluster = 1;  // more blocks while they would be idle and a block has several rounds of pages
    while (cluster < 8 && 2LL * cluster * units <= 2LL * n_sm && p.t.max_pages > cluster * (kSelectThreads / 4)) cluster *= 2;
    const int smem = 4 * p.t.max_pages;
    auto go = [&](auto* f) {
        const cudaError_t e = smem_opt_in(reinterpret_cast<const void*>(f), 4 * kSelectMostPages);
        return e != cudaSuccess ? e : launch_cluster(f, units * cluster, cluster, kSelectThreads, smem, stream, p);
    };
    return p.c.d == 64 ? go(select_kernel<64>) : go(select_kernel<128>);
}

}  // namespace attn
