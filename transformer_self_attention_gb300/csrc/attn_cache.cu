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
// Bound by memory: each row is read once and written once.  The mapping of rows to threads is rope_kernel's
// (attn_rope.cu): d / 16 threads hold a row, 16 elements each, and a thread walks over the heads of one token,
// queries, keys and values in one list.
#include <cuda_runtime.h>

#include <algorithm>

#include "paged.h"
#include "sm103_ptx.h"

namespace attn {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float exponent_factor(int e) {  // 2^(e - 127); NaN for 255
    return __uint_as_float(e == 0 ? 0x00400000u : e == 255 ? 0x7FFFFFFFu : (uint32_t)e << 23);
}
// The exponent k of a row whose largest magnitude is `big` (finite): 448 = 1.75 * 2^8.
__device__ __forceinline__ int row_exponent(float big) {
    const uint32_t w = __float_as_uint(big);
    const int k = (int)(w >> 23) - 127 - 8 + ((w & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return max(k, -127);
}

struct WriteLaunch {
    CacheWriteParams p;
    int tb, hb, heads_block, tokens;
};

template <int D, bool E4M3, bool STAGED>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const __grid_constant__ WriteLaunch a) {
    constexpr int LANES = D / 16;
    __shared__ unsigned long long step[D / 2];
    __shared__ float stage[STAGED ? kThreads / LANES * (D + 1) : 1];
    const CacheWriteParams& p = a.p;
    const int u = threadIdx.x % LANES, slot = threadIdx.x / LANES;
    const int token = blockIdx.x * a.tb + slot / a.hb;
    const bool live = slot < a.tb * a.hb && token < a.tokens;
    const int b = live ? token / p.S : 0, i = live ? token - b * p.S : 0;
    const bool halves = !p.rope.interleaved;
    int off_a = 16 * u, off_b = 16 * u + 8;
    if (!STAGED) rope_runs(halves, p.rope.rot, u, off_a, off_b);
    const bool across = !STAGED && halves && 16 * u < p.rope.rot;
    const int H = p.Hq + 2 * p.c.Hkv;
    const int h_first = blockIdx.y * a.heads_block, h_last = min(H, h_first + a.heads_block);
    constexpr int U = STAGED ? 1 : 2;
    // The next U rows, on their way before what they need is known (rows of padding are read too, and not used).
    Raw8<__nv_bfloat16> raw[U][2];
    auto fetch = [&](int h0) {
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int h = h0 + j * a.hb + slot % a.hb;
            if (!live || h >= h_last) continue;
            const int kind = h < p.Hq ? 1 : h < p.Hq + p.c.Hkv ? 2 : 3;
            const RopeRows& r = kind == 1 ? p.q : kind == 2 ? p.k : p.v;
            const int head = h - (kind == 1 ? 0 : kind == 2 ? p.Hq : p.Hq + p.c.Hkv);
            const __nv_bfloat16* in = reinterpret_cast<const __nv_bfloat16*>(r.src) + (b * r.sb + head * r.sh + i * r.ss);
            const bool apart = across && kind != 3;
            fetch8(in + (apart ? off_a : 16 * u), raw[j][0]);
            fetch8(in + (apart ? off_b : 16 * u + 8), raw[j][1]);
        }
    };
    fetch(h_first);
    const int len = p.t.len[b];
    const int fresh = p.new_len ? p.new_len[b] : p.S;
    const int pos = len - fresh + i;
    const bool valid = live && i < fresh && pos >= 0;  // a sequence shorter than its rows: padding in front
    // where the token's rows go; a bad one is recorded and skipped
    bool placed = false;
    int page = 0, in_page = 0;
    if (valid) {
        int bad = 0;
        if (pos >= (long long)p.t.max_pages * p.c.page) {
            bad = kCacheErrPosition;
        } else {
            page = p.t.pages[b * p.t.stride + pos / p.c.page];
            in_page = pos % p.c.page;
            if (page < 0 || page >= p.c.n_pages) bad = kCacheErrPage;
        }
        placed = bad == 0;
        if (bad && u == 0) atomicOr(p.c.err, bad);
    }
    if ((int)threadIdx.x < p.rope.rot / 2) step[threadIdx.x] = p.rope.step[threadIdx.x];
    __syncthreads();
    float c[8], sn[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int q = 8 * u + e;
        c[e] = 1.f;
        sn[e] = 0.f;
        if (2 * q < p.rope.rot) {
            rope_cos_sin(pos, step[q], c[e], sn[e]);
            c[e] *= p.rope.amp;
            sn[e] *= p.rope.amp;
        }
    }
    for (int h0 = h_first; h0 < h_last; h0 += U * a.hb) {
        float run[U][16];
        int what[U], head[U];  // 0: nothing, 1: a query, 2: a key, 3: a value
        bool swap[U];          // the lane's runs are the two halves of pairs
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int h = h0 + j * a.hb + slot % a.hb;
            what[j] = !live || h >= h_last ? 0 : h < p.Hq ? 1 : h < p.Hq + p.c.Hkv ? 2 : 3;
            head[j] = h - (what[j] == 1 ? 0 : what[j] == 2 ? p.Hq : p.Hq + p.c.Hkv);
            swap[j] = across && what[j] != 3;
            widen8(raw[j][0], run[j]);
            widen8(raw[j][1], run[j] + 8);
            if (what[j] == 0 || !valid)
#pragma unroll
                for (int e = 0; e < 16; ++e) run[j][e] = 0.f;
        }
        fetch(h0 + U * a.hb);
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if (STAGED) {  // pairs of halves off the 8-element grid: through shared memory, within the row's warp
                float* row = stage + slot * (D + 1);
                float x[16];
                __syncwarp();
#pragma unroll
                for (int e = 0; e < 16; ++e) row[16 * u + e] = run[j][e];
                __syncwarp();
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    int i0, i1;
                    rope_pair_index(halves, p.rope.rot, 8 * u + e, i0, i1);
                    x[2 * e] = row[i0];
                    x[2 * e + 1] = row[i1];
                }
                if (what[j] != 3) rope_turn(x, c, sn);
                __syncwarp();
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    int i0, i1;
                    rope_pair_index(halves, p.rope.rot, 8 * u + e, i0, i1);
                    row[i0] = x[2 * e];
                    row[i1] = x[2 * e + 1];
                }
                __syncwarp();
#pragma unroll
                for (int e = 0; e < 16; ++e) run[j][e] = row[16 * u + e];
            } else if (what[j] == 1 || what[j] == 2) {
                float x[16];
                runs_to_pairs(swap[j], run[j], run[j] + 8, x);
                rope_turn(x, c, sn);
                pairs_to_runs(swap[j], x, run[j], run[j] + 8);
            }
            float big = 0.f;
            bool odd = false;  // an infinity or a NaN in the row
            if (E4M3) {
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float m = fabsf(run[j][e]);
                    big = fmaxf(big, m);
                    odd |= !(m <= 3.402823466e38f);
                }
                // the lanes of a row: LANES neighbours, on a multiple of LANES
#pragma unroll
                for (int o = LANES / 2; o; o >>= 1) {
                    big = fmaxf(big, __shfl_xor_sync(0xFFFFFFFFu, big, o));
                    odd |= __shfl_xor_sync(0xFFFFFFFFu, (int)odd, o) != 0;
                }
            }
            const int ra = swap[j] ? off_a : 16 * u, rb = swap[j] ? off_b : 16 * u + 8;
            if (what[j] == 1) {
                __nv_bfloat16* out =
                    reinterpret_cast<__nv_bfloat16*>(p.q.dst) + (b * p.q.db + head[j] * p.q.dh + i * p.q.ds);
                store8(out + ra, run[j]);
                store8(out + rb, run[j] + 8);
            } else if (what[j] >= 2 && placed) {
                const long long unit = (long long)page * p.c.Hkv + head[j];
                const int kv = what[j] - 2;
                const long long row = (unit * 2 + kv) * p.c.page + in_page;
                if (E4M3) {
                    const int k = odd ? 128 : row_exponent(big);
                    const float f = exponent_factor(max(0, 127 - k));  // 2^-k
                    uint32_t w[4];
#pragma unroll
                    for (int g = 0; g < 4; ++g)
                        w[g] = odd ? 0x7F7F7F7Fu
                                   : ptx::pack_e4m3x4(run[j][4 * g] * f, run[j][4 * g + 1] * f, run[j][4 * g + 2] * f,
                                                      run[j][4 * g + 3] * f);
                    char* out = p.c.pages + row * D;
                    *reinterpret_cast<uint2*>(out + ra) = make_uint2(w[0], w[1]);
                    *reinterpret_cast<uint2*>(out + rb) = make_uint2(w[2], w[3]);
                    if (u == 0)
                        p.c.scales[((unit * (p.c.page / 16) + in_page / 16) * 2 + kv) * 16 + in_page % 16] =
                            (uint8_t)(k + 127);
                } else {
                    __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(p.c.pages) + row * D;
                    store8(out + ra, run[j]);
                    store8(out + rb, run[j] + 8);
                }
            }
        }
    }
}

// Readback: each D / 16 threads take one (position, kv head, K or V) row.  Rows at or past the length are left as they
// are.  E4M3 codes become fp16 (exact), then times 2^k, which bf16 holds exactly.
template <int D, bool E4M3>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const __grid_constant__ CacheReadParams p) {
    constexpr int LANES = D / 16, ROWS = kThreads / LANES;
    const int u = threadIdx.x % LANES, slot = threadIdx.x / LANES;
    const int s = blockIdx.x * ROWS + slot, b = blockIdx.z;
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

int pow2_at_least(int n) {
    int p = 1;
    while (p < n) p *= 2;
    return p;
}

template <int D, bool E4M3>
cudaError_t write_d(const CacheWriteParams& p, int n_sm, cudaStream_t stream) {
    WriteLaunch a{};
    a.p = p;
    a.tokens = p.B * p.S;
    const int rows = kThreads / (D / 16), H = p.Hq + 2 * p.c.Hkv;
    const int heads = std::min(8, pow2_at_least(H / 8 / 2 + 1));  // side by side, as in launch_rope
    a.tb = std::min(rows / heads, pow2_at_least(a.tokens));
    a.hb = rows / a.tb;
    const long long blocks_x = (a.tokens + (long long)a.tb - 1) / a.tb;
    const int rounds = (H + a.hb - 1) / a.hb;
    const long long want = 4LL * n_sm;
    const int split = (int)std::min<long long>(rounds, std::max<long long>(1, (want + blocks_x - 1) / blocks_x));
    a.heads_block = (rounds + split - 1) / split * a.hb;
    const dim3 grid((unsigned)blocks_x, (unsigned)((H + a.heads_block - 1) / a.heads_block));
    if (!p.rope.interleaved && p.rope.rot % 16 != 0)
        cache_write_kernel<D, E4M3, true><<<grid, kThreads, 0, stream>>>(a);
    else
        cache_write_kernel<D, E4M3, false><<<grid, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

template <int D, bool E4M3>
cudaError_t read_d(const CacheReadParams& p, cudaStream_t stream) {
    const int rows = kThreads / (D / 16);
    const unsigned gx = (unsigned)((p.S + rows - 1) / rows);
    const dim3 grid(gx, (unsigned)std::min(p.c.Hkv, 65535), (unsigned)p.B);
    cache_read_kernel<D, E4M3><<<grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
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
