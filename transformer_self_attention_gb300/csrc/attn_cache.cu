// The paged key/value cache: rows written into pages, and positions read back.
//
// Write.  Row i of sequence b goes to position t = len[b] - new_len[b] + i: slot t % page of the page
// table[b, t / page].  Keys are rotated on the way (and the queries of the same tokens with them), so that a
// rotated key is rounded once, to what the cache holds.  E4M3 rows x are held as codes and one exponent:
//     k = min { k : max|x| 2^-k <= 448 },   code = rn_e4m3(x 2^-k),   the row stands for code * 2^k.
// A power of two costs a float code no relative precision, makes x 2^-k, the product in the decode
// kernel and the readback to bf16 exact, and takes one byte.  A row with an infinity or a NaN gets NaN codes and
// exponent byte 255: it reads back as NaN throughout.
//
// Bound by memory: each row is read once and written once.  d / 16 lanes hold a row, 16 elements each (attn_rope.cu),
// and a warp takes one token after another, two rows a lane: 7.1K tokens of 8 heads to E4M3, keys rotated, take 15 us
// (2.9 TB/s; the smaller the chunk, the more the first loads' latency counts), 50.6K tokens of 8 heads to bf16 72 us (5.7
// TB/s, 85% of the measured copy rate) and to E4M3 81 us (3.9 TB/s; instructions: 0.7 a clock).  Blocks whose warps shared
// their tokens by way of shared memory were no faster.
#include <cuda_runtime.h>

#include <algorithm>

#include "paged_device.h"

namespace attn {

namespace {

constexpr int kThreads = 256;
// Of the write kernel, which hides its loads behind its arithmetic: five blocks of 128 threads (96 registers a thread) a
// multiprocessor took 68 us for 48.5K bf16 tokens, four 74.
constexpr int kWriteThreads = 128, kWriteBlocks = 5;

__device__ __forceinline__ float exponent_factor(int e) {  // 2^(e - 127); NaN for 255
    return __uint_as_float(e == 0 ? 0x00400000u : e == 255 ? 0x7FFFFFFFu : (uint32_t)e << 23);
}
// The exponent k of a row whose largest magnitude is `big` (finite): 448 = 1.75 * 2^8.
__device__ __forceinline__ int row_exponent(float big) {
    const uint32_t w = __float_as_uint(big);
    const int k = (int)(w >> 23) - 127 - 8 + ((w & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return max(k, -127);
}

// x / n for 0 <= x < 2^31 by a multiplication: mul = ceil(2^(31 + shift) / n) with 2^shift >= n (exact for 31-bit x).
struct Divisor {
    unsigned n = 1, mul = 0, shift = 0;
    Divisor() = default;
    explicit Divisor(unsigned n_) : n(n_) {
        while ((1ull << shift) < n) ++shift;
        mul = (unsigned)(((1ull << (31 + shift)) + n - 1) / n);
    }
    __device__ __forceinline__ int div(int x) const {
        return (int)(((unsigned long long)(unsigned)x * mul) >> (31 + shift));
    }
};

struct WriteLaunch {
    CacheWriteParams p;
    int tokens, items, chunks, items_chunk;  // items of a token: two queries, or a key and its value
    Divisor by_S, by_page, by_chunks;
};

// Largest of |x| and y; NaN if either is one.
__device__ __forceinline__ float max_abs_nan(float x, float y) {
    float z;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(fabsf(x)), "f"(y));
    return z;
}

// Turns the lane's runs of a row, through shared memory where the pairs do not sit on the 8-element grid (STAGED).
template <bool HALVES, bool STAGED>
__device__ __forceinline__ void turn_row(float (&run)[16], float* row, int rot, int u, const float (&c)[8],
                                         const float (&s)[8], int live) {
    if (!STAGED) {
        rope_turn<HALVES>(run, c, s, live);
        return;
    }
    float x[16];
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 16; ++e) row[16 * u + e] = run[e];
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        int i0, i1;
        rope_pair_index(HALVES, rot, 8 * u + e, i0, i1);
        x[2 * e] = row[i0];
        x[2 * e + 1] = row[i1];
    }
    rope_turn<false>(x, c, s, live);
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        int i0, i1;
        rope_pair_index(HALVES, rot, 8 * u + e, i0, i1);
        row[i0] = x[2 * e];
        row[i1] = x[2 * e + 1];
    }
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 16; ++e) run[e] = row[16 * u + e];
}

// HALVES: the rotated pairs are (p, p + rot / 2), otherwise neighbours.  STAGED: pairs of halves off the 8-element grid.
// QUERIES: there may be some (without, fewer registers).
// A thread takes two rows at a time: two queries, or a head's key and value.  (One row at a time, with its kind and place
// found anew, took 300 instructions a row and 103 us for 48.5K tokens of 8 heads, 4 TB/s.)
template <int D, bool E4M3, bool HALVES, bool STAGED, bool QUERIES>
__global__ void __launch_bounds__(kWriteThreads, kWriteBlocks) cache_write_kernel(const __grid_constant__ WriteLaunch a) {
    constexpr int LANES = D / 16, SLOTS = 32 / LANES, WARPS = kWriteThreads / 32;
    __shared__ float2 turns[WARPS][D / 2];
    __shared__ unsigned long long step[D / 2];
    __shared__ float stage[STAGED ? WARPS * SLOTS * (D + 1) : 1];
    const CacheWriteParams& p = a.p;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, u = lane % LANES, slot = lane / LANES;
    const int pairs = p.rope.rot / 2, live = rope_live_pairs(u, p.rope.rot), q_items = QUERIES ? (p.Hq + 1) / 2 : 0;
    int off_a = 16 * u, off_b = 16 * u + 8;
    if (!STAGED) rope_runs(HALVES, p.rope.rot, u, off_a, off_b);
    typedef const __nv_bfloat16* Src;

    // A warp takes one token's items (a chunk of them where there are few tokens) after another; what the next step needs
    // is always on its way.
    struct Job {
        int token, b, i, fresh, item, end;  // item: the lane's next; end: behind the chunk
        int pos, entry, slot;               // position (-1: padding), its page-table entry and slot
    };
    auto open = [&](int job) {
        Job j;
        j.token = a.by_chunks.div(job);
        const int chunk = job - j.token * a.chunks;
        j.item = chunk * a.items_chunk + slot;
        j.end = min(a.items, (chunk + 1) * a.items_chunk);
        j.b = a.by_S.div(j.token);
        j.i = j.token - j.b * p.S;
        j.fresh = p.new_len ? p.new_len[j.b] : p.S;
        j.pos = p.t.len[j.b] - j.fresh + j.i;
        j.entry = -1;
        j.slot = 0;
        if (j.i >= j.fresh || j.pos < 0) {
            j.pos = -1;  // padding; also in front of a sequence shorter than its rows
        } else if (j.pos >= (long long)p.t.max_pages * p.c.page) {
            j.entry = -2;
        } else {
            const int index = a.by_page.div(j.pos);
            j.slot = j.pos - index * p.c.page;
            j.entry = p.t.pages[j.b * p.t.stride + index];
        }
        return j;
    };
    Raw8<__nv_bfloat16> raw[2][2] = {};
    auto fetch = [&](const Job& j, int item) {
        if (item >= j.end || j.i >= j.fresh) return;  // rows of padding are not read
        const bool query = QUERIES && item < q_items;
        const int h = query ? 2 * item : item - q_items;
        const RopeRows& r = query ? p.q : p.k;
        const Src r0 = reinterpret_cast<Src>(r.src) + (j.b * r.sb + j.i * r.ss + h * r.sh);
        fetch8(r0 + off_a, raw[0][0]);
        fetch8(r0 + off_b, raw[0][1]);
        if (query) {
            if (h + 1 < p.Hq) {
                fetch8(r0 + p.q.sh + off_a, raw[1][0]);
                fetch8(r0 + p.q.sh + off_b, raw[1][1]);
            }
        } else {
            const Src r1 = reinterpret_cast<Src>(p.v.src) + (j.b * p.v.sb + j.i * p.v.ss + h * p.v.sh) + 16 * u;
            fetch8(r1, raw[1][0]);
            fetch8(r1 + 8, raw[1][1]);
        }
    };
    wait_for_kernel_before();
    let_kernel_behind_in();
    // (the frequencies lie in the parameters, where 32 different words take 32 reads)
    if ((int)threadIdx.x < pairs) step[threadIdx.x] = p.rope.step[threadIdx.x];
    __syncthreads();
    const int jobs = a.tokens * a.chunks, stride = gridDim.x * WARPS;
    int job = blockIdx.x * WARPS + warp;
    if (job >= jobs) return;
    Job now = open(job);
    fetch(now, now.item);
    for (; job < jobs; job += stride) {
        Job next = now;
        const bool more = job + stride < jobs;
        if (more) next = open(job + stride);
        for (int q = lane; q < pairs; q += 32) {
            float cq, sq;
            rope_cos_sin(now.pos, step[q], cq, sq);
            turns[warp][q] = make_float2(cq * p.rope.amp, sq * p.rope.amp);
        }
        __syncwarp();
        float c[8], sn[8];
        rope_lane_turns(turns[warp], u, p.rope.rot, c, sn);
        __syncwarp();
        struct {
            int pos, page, slot;
        } at{now.pos, now.entry, now.slot};
        if (at.pos >= 0 && (at.page < 0 || at.page >= p.c.n_pages)) {  // a bad place is recorded and skipped
            const bool beyond = at.pos >= (long long)p.t.max_pages * p.c.page;
            if (lane == 0) atomicOr(p.c.err, beyond ? kCacheErrPosition : kCacheErrPage);
            at.page = -1;
        }
        const int b = now.b, i = now.i;
        // the token's slot in kv head 0 of its page, and the bytes from one head to the next
        constexpr int kRow = D * (E4M3 ? 1 : 2);
        const long long head_bytes = 2LL * p.c.page * kRow;
        char* const keys = p.c.pages + (long long)at.page * p.c.Hkv * head_bytes + at.slot * kRow;
        for (int item = now.item; __any_sync(0xFFFFFFFFu, item < now.end); item += SLOTS) {
            float run[2][16];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                widen8(raw[j][0], run[j]);
                widen8(raw[j][1], run[j] + 8);
            }
            const bool last = !__any_sync(0xFFFFFFFFu, item + SLOTS < now.end);
            if (!last) fetch(now, item + SLOTS);
            else if (more) fetch(next, next.item);
            const bool query = QUERIES && item < q_items;
            float* const row = stage + (STAGED ? (warp * SLOTS + slot) * (D + 1) : 0);
            turn_row<HALVES, STAGED>(run[0], row, p.rope.rot, u, c, sn, live);
            float second[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) second[e] = run[1][e];
            if (QUERIES) turn_row<HALVES, STAGED>(second, row, p.rope.rot, u, c, sn, live);
            float big[2] = {0.f, 0.f};
            if (E4M3) {
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    big[0] = max_abs_nan(run[0][e], big[0]);
                    big[1] = max_abs_nan(run[1][e], big[1]);
                }
                // the lanes of a row: LANES neighbours, on a multiple of LANES
#pragma unroll
                for (int o = LANES / 2; o; o >>= 1)
#pragma unroll
                    for (int j = 0; j < 2; ++j) big[j] = max_abs_nan(__shfl_xor_sync(0xFFFFFFFFu, big[j], o), big[j]);
            }
            if (item >= now.end) continue;
            if (query) {
                const int h = 2 * item;
                __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(p.q.dst) + (b * p.q.db + h * p.q.dh + i * p.q.ds);
                if (at.pos < 0)
#pragma unroll
                    for (int e = 0; e < 16; ++e) run[0][e] = second[e] = 0.f;
                store8(out + off_a, run[0]);
                store8(out + off_b, run[0] + 8);
                if (h + 1 < p.Hq) {
                    store8(out + p.q.dh + off_a, second);
                    store8(out + p.q.dh + off_b, second + 8);
                }
            } else if (at.page >= 0) {
                const int h = item - q_items;
                char* const key = keys + h * head_bytes;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    char* const out = key + j * (head_bytes / 2);
                    const int ra = j ? 16 * u : off_a, rb = j ? 16 * u + 8 : off_b;
                    if (E4M3) {
                        const bool odd = !(big[j] <= 3.402823466e38f);  // an infinity or a NaN in the row
                        const int k = odd ? 128 : row_exponent(big[j]);
                        const float f = exponent_factor(max(0, 127 - k));  // 2^-k
                        uint32_t w[4];
#pragma unroll
                        for (int g = 0; g < 4; ++g)
                            w[g] = odd ? 0x7F7F7F7Fu
                                       : ptx::pack_e4m3x4(run[j][4 * g] * f, run[j][4 * g + 1] * f, run[j][4 * g + 2] * f,
                                                          run[j][4 * g + 3] * f);
                        *reinterpret_cast<uint2*>(out + ra) = make_uint2(w[0], w[1]);
                        *reinterpret_cast<uint2*>(out + rb) = make_uint2(w[2], w[3]);
                        if (u == 0) {
                            const long long unit = (long long)at.page * p.c.Hkv + h;
                            const long long at16 = (unit * (p.c.page / 16) + at.slot / 16) * 2 + j;
                            p.c.scales[at16 * 16 + at.slot % 16] = (uint8_t)(k + 127);
                        }
                    } else {
                        store8(reinterpret_cast<__nv_bfloat16*>(out) + ra, run[j]);
                        store8(reinterpret_cast<__nv_bfloat16*>(out) + rb, run[j] + 8);
                    }
                }
            }
        }
        now = next;
    }
}

// Readback: each D / 16 threads take one (position, kv head, K or V) row.  Many small blocks hide the three dependent loads
// (length, page, row): 21.6K ragged positions of 8 heads, E4M3 (133 MB), take 26.0 us, 75% of the measured copy rate (bf16,
// 177 MB, 28.8 us, 91%); two and four heads a thread with all loads first took 29.0 and 29.8.  Rows at or past the length
// are left as they are.  E4M3 codes
// become fp16 (exact), then times 2^k, which bf16 holds exactly.
template <int D, bool E4M3>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const __grid_constant__ CacheReadParams p) {
    constexpr int LANES = D / 16, ROWS = kThreads / LANES;
    const int u = threadIdx.x % LANES, slot = threadIdx.x / LANES;
    const int s = blockIdx.x * ROWS + slot, b = blockIdx.z;
    wait_for_kernel_before();
    let_kernel_behind_in();
    if (s >= p.S) return;
    const long long pos = (long long)p.first + s;
    const int len = p.t.len[b];
    const long long room = (long long)p.t.max_pages * p.c.page;
    if ((len < 0 || len > room) && s == 0 && u == 0) atomicOr(p.c.err, kCacheErrPosition);
    if (pos >= len || pos >= room) return;
    const int page = p.t.pages[b * p.t.stride + pos / p.c.page], in_page = (int)(pos % p.c.page);
    if (page < 0 || page >= p.c.n_pages) {
        if (u == 0) atomicOr(p.c.err, kCacheErrPage);
        return;
    }
    for (int h = blockIdx.y; h < p.c.Hkv; h += gridDim.y) {
        const long long unit = (long long)page * p.c.Hkv + h;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            const long long row = (unit * 2 + kv) * p.c.page + in_page;
            const RopeRows& r = kv == 0 ? p.k : p.v;
            __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(r.dst) + (b * r.db + h * r.dh + s * r.ds) + 16 * u;
            if (E4M3) {
                const uint4 v = *reinterpret_cast<const uint4*>(p.c.pages + row * D + 16 * u);
                const float f = exponent_factor(
                    p.c.scales[((unit * (p.c.page / 16) + in_page / 16) * 2 + kv) * 16 + in_page % 16]);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                float x[16];
#pragma unroll
                for (int g = 0; g < 4; ++g) {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t two;
                        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(two) : "h"((uint16_t)(w[g] >> (16 * half))));
                        float lo, hi;
                        asm("{.reg .f16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b;}"
                            : "=f"(lo), "=f"(hi)
                            : "r"(two));
                        x[4 * g + 2 * half] = lo * f;
                        x[4 * g + 2 * half + 1] = hi * f;
                    }
                }
                store8(out, x);
                store8(out + 8, x + 8);
            } else {
                const uint4* in = reinterpret_cast<const uint4*>(p.c.pages + row * D * 2) + 2 * u;
                const uint4 v0 = in[0], v1 = in[1];
                reinterpret_cast<uint4*>(out)[0] = v0;
                reinterpret_cast<uint4*>(out)[1] = v1;
            }
        }
    }
}

template <int D, bool E4M3>
cudaError_t write_d(const CacheWriteParams& p, int n_sm, cudaStream_t stream) {
    WriteLaunch a{};
    a.p = p;
    a.tokens = p.B * p.S;
    a.items = (p.Hq + 1) / 2 + p.c.Hkv;
    a.by_S = Divisor(p.S);
    a.by_page = Divisor(p.c.page);
    // a warp takes all items of a token unless that leaves multiprocessors without their warps
    const int slots = 32 / (D / 16), rounds = (a.items + slots - 1) / slots, warps = kWriteThreads / 32;
    const long long want = (long long)kWriteBlocks * warps * n_sm;
    const int split = (int)std::min<long long>(rounds, std::max<long long>(1, (want + a.tokens - 1) / a.tokens));
    a.items_chunk = (rounds + split - 1) / split * slots;
    a.chunks = (a.items + a.items_chunk - 1) / a.items_chunk;
    a.by_chunks = Divisor(a.chunks);
    const long long blocks = ((long long)a.tokens * a.chunks + warps - 1) / warps;
    const unsigned grid = (unsigned)std::min<long long>(blocks, (long long)kWriteBlocks * n_sm);
    auto go = [&](auto* f) { return launch_dependent(f, dim3(grid), kWriteThreads, 0, stream, a); };
    const bool q = p.Hq > 0;
    if (p.rope.interleaved)
        return q ? go(cache_write_kernel<D, E4M3, false, false, true>) : go(cache_write_kernel<D, E4M3, false, false, false>);
    if (p.rope.rot % 16 != 0) return go(cache_write_kernel<D, E4M3, true, true, true>);
    return q ? go(cache_write_kernel<D, E4M3, true, false, true>)
             : go(cache_write_kernel<D, E4M3, true, false, false>);
}

template <int D, bool E4M3>
cudaError_t read_d(const CacheReadParams& p, cudaStream_t stream) {
    const int rows = kThreads / (D / 16);
    const unsigned gx = (unsigned)((p.S + rows - 1) / rows);
    const dim3 grid(gx, (unsigned)std::min(p.c.Hkv, 65535), (unsigned)p.B);
    return launch_dependent(cache_read_kernel<D, E4M3>, grid, kThreads, 0, stream, p);
}

}  // namespace

cudaError_t launch_cache_write(const CacheWriteParams& p, bool e4m3, int n_sm, cudaStream_t stream) {
    if (p.c.d == 64) return e4m3 ? write_d<64, true>(p, n_sm, stream) : write_d<64, false>(p, n_sm, stream);
    return e4m3 ? write_d<128, true>(p, n_sm, stream) : write_d<128, false>(p, n_sm, stream);
}
cudaError_t launch_cache_read(const CacheReadParams& p, bool e4m3, cudaStream_t stream) {
    if (p.c.d == 64) return e4m3 ? read_d<64, true>(p, stream) : read_d<64, false>(p, stream);
    return e4m3 ? read_d<128, true>(p, stream) : read_d<128, false>(p, stream);
}

}  // namespace attn
