// Rotary positions applied to the rows of Q and K, and the gradient of that rotation.
//
//     (x_p, x_p') -> amp (x_p cos t - x_p' sin t,  x_p sin t + x_p' cos t),  t = f_p * position,
//
// over the rot / 2 pairs of a row; the d - rot elements behind them are copied.  The gradient is the transpose:
// the same with -t.  Bound by memory: every element is read once and written once, about 3 flops each.
//
// A row is held by d / 16 neighbouring threads, 16 elements each, as two 16-byte runs of bf16 (four of fp32), so
// that the loads and stores of a warp cover whole rows.  A thread keeps one token and walks over heads.  The cosines and
// sines of a block's tokens (about 45 instructions each) are computed once, into shared memory.
#include <cuda_runtime.h>

#include <algorithm>

#include "paged_device.h"

namespace attn {

namespace {

constexpr int kThreads = 256;

struct RopeParams {
    RopeTable t;
    RopeRows q, k;
    int Hq, H;  // query heads; query and key heads
    int S, tokens, d;
    int tb, hb;       // tokens and heads of a block side by side: tb * hb rows
    int heads_block;  // heads a block walks over
    const int* positions;
    long long pos_b, pos_s;
    float sign;  // -1: the gradient
    int warp_rows;  // no row spans two warps
};

// Orders the shared-memory accesses of a row's threads.
__device__ __forceinline__ void row_sync(int warp_rows) {
    if (warp_rows) __syncwarp();
    else __syncthreads();
}

// U rows a thread are fetched before the cosines and sines are computed, and the next U before the present ones are
// turned, so that loads are always under way.
// STAGED: pairs of halves whose second half does not start on an 8-element boundary.  The row goes through shared
// memory, where the pairs are picked element by element; global accesses stay 16 bytes wide.
// Three blocks of bf16 rows a multiprocessor: with two, 8K tokens of 64 heads take 51.4 us for 45.2.
template <class T, bool HALVES, bool STAGED, int U>
__global__ void __launch_bounds__(kThreads, (sizeof(T) == 2 ? 3 : 2)) rope_kernel(const __grid_constant__ RopeParams p) {
    extern __shared__ uint32_t stage[];
    __shared__ float2 turns[kThreads * 8];  // rows of a block * rot / 2 at most
    __shared__ unsigned long long step[kRopeMaxPairs];
    const int lanes = p.d / 16, u = threadIdx.x % lanes, slot = threadIdx.x / lanes;
    const int token = blockIdx.x * p.tb + slot / p.hb;
    const bool live = slot < p.tb * p.hb && token < p.tokens;
    const int b = live ? token / p.S : 0, s = live ? token - b * p.S : 0;
    int off_a = 16 * u, off_b = 16 * u + 8;
    if (!STAGED) rope_runs(HALVES, p.t.rot, u, off_a, off_b);
    const int h_first = blockIdx.y * p.heads_block, h_last = min(p.H, h_first + p.heads_block);

    Raw8<T> raw[U][2];
    auto fetch = [&](int h0) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int h = h0 + i * p.hb + slot % p.hb;
            if (!live || h >= h_last) continue;
            const RopeRows& r = h < p.Hq ? p.q : p.k;
            const T* in = reinterpret_cast<const T*>(r.src) + (b * r.sb + (h < p.Hq ? h : h - p.Hq) * r.sh + s * r.ss);
            fetch8(in + off_a, raw[i][0]);
            fetch8(in + off_b, raw[i][1]);
        }
    };
    wait_for_kernel_before();
    let_kernel_behind_in();
    fetch(h_first);
    // (the frequencies lie in the parameters, where 32 different words take 32 reads)
    const int pairs = p.t.rot / 2;
    if ((int)threadIdx.x < pairs) step[threadIdx.x] = p.t.step[threadIdx.x];
    __syncthreads();
    for (int i = threadIdx.x; i < p.tb * pairs; i += kThreads) {
        const int q = i % pairs, t = min((int)blockIdx.x * p.tb + i / pairs, p.tokens - 1);
        const int tb = t / p.S, ts = t - tb * p.S;
        const int pos = p.positions ? p.positions[tb * p.pos_b + ts * p.pos_s] : ts;
        float cq, sq;
        rope_cos_sin(pos, step[q], cq, sq);
        turns[i] = make_float2(cq * p.t.amp, sq * (p.t.amp * p.sign));
    }
    __syncthreads();
    float c[8], sn[8];
    const int live_pairs = rope_live_pairs(u, p.t.rot);
    rope_lane_turns(turns + min(slot / p.hb, p.tb - 1) * pairs, u, p.t.rot, c, sn);
    for (int h0 = h_first; h0 < h_last; h0 += U * p.hb) {
        float run[U][16];
        Raw8<T> raw_now[U][2];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (STAGED) {
                raw_now[i][0] = raw[i][0];
                raw_now[i][1] = raw[i][1];
            } else {
                widen8(raw[i][0], run[i]);
                widen8(raw[i][1], run[i] + 8);
            }
        }
        fetch(h0 + U * p.hb);
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int h = h0 + i * p.hb + slot % p.hb;
            const bool row_live = live && h < h_last;
            if (STAGED) {
                // Word by word, rows one word apart in the banks: at most two lanes of a warp meet in a bank.
                constexpr int kWords = 16 * sizeof(T) / 4;
                const bool on = slot < p.tb * p.hb;
                uint32_t* row = stage + slot * (p.d * (int)sizeof(T) / 4 + 1);
                T* row_t = reinterpret_cast<T*>(row);
                const uint32_t* mine = reinterpret_cast<const uint32_t*>(raw_now[i]);
                row_sync(p.warp_rows);
                if (on)
#pragma unroll
                    for (int e = 0; e < kWords; ++e) row[kWords * u + e] = mine[e];
                row_sync(p.warp_rows);
                float x[16];
                if (on) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        int i0, i1;
                        rope_pair_index(HALVES, p.t.rot, 8 * u + e, i0, i1);
                        x[2 * e] = (float)row_t[i0];
                        x[2 * e + 1] = (float)row_t[i1];
                    }
                    rope_turn<false>(x, c, sn, live_pairs);
                }
                row_sync(p.warp_rows);
                if (on)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        int i0, i1;
                        rope_pair_index(HALVES, p.t.rot, 8 * u + e, i0, i1);
                        row_t[i0] = (T)x[2 * e];
                        row_t[i1] = (T)x[2 * e + 1];
                    }
                row_sync(p.warp_rows);
                if (!row_live) continue;
                const RopeRows& r = h < p.Hq ? p.q : p.k;
                uint4* out = reinterpret_cast<uint4*>(reinterpret_cast<T*>(r.dst) +
                                                      (b * r.db + (h < p.Hq ? h : h - p.Hq) * r.dh + s * r.ds) + 16 * u);
#pragma unroll
                for (int e = 0; e < kWords; e += 4)
                    out[e / 4] = make_uint4(row[kWords * u + e], row[kWords * u + e + 1], row[kWords * u + e + 2],
                                            row[kWords * u + e + 3]);
                continue;
            } else {
                rope_turn<HALVES>(run[i], c, sn, live_pairs);
            }
            if (!row_live) continue;
            const RopeRows& r = h < p.Hq ? p.q : p.k;
            T* out = reinterpret_cast<T*>(r.dst) + (b * r.db + (h < p.Hq ? h : h - p.Hq) * r.dh + s * r.ds);
            store8(out + off_a, run[i]);
            store8(out + off_b, run[i] + 8);
        }
    }
}

int pow2_at_least(int n) {
    int p = 1;
    while (p < n) p *= 2;
    return p;
}

}  // namespace

cudaError_t launch_rope(const RopeTable& t, const RopeRows& q, const RopeRows& k, int Hq, int Hk, int B, int S, int d,
                        const int* positions, long long pos_b, long long pos_s, bool inverse, bool f32, int n_sm,
                        cudaStream_t stream) {
    RopeParams p{};
    p.t = t;
    p.q = q;
    p.k = k;
    p.Hq = Hq;
    p.H = Hq + Hk;
    p.S = S;
    p.tokens = B * S;
    p.d = d;
    p.positions = positions;
    p.pos_b = pos_b;
    p.pos_s = pos_s;
    p.sign = inverse ? -1.f : 1.f;
    const int rows = kThreads / (d / 16);
    const int heads_wide = p.H >= 64 ? 8 : 4;
    p.warp_rows = 32 % (d / 16) == 0;
    // Four or eight heads side by side (their rows are neighbours in a [B, S, H, d] projection), so that a thread still
    // walks over eight or so; the other rows of a block are neighbouring tokens (neighbours in [B, H, S, d]); few tokens
    // leave more rows to the heads.  With 2, 4, 8, 16 heads side by side: 64 heads x 8K tokens 49.8, 46.8, 44.6, 47.0 us,
    // 40 heads x 16K tokens 57.9, 55.2, 58.8, 70.3 us.
    p.tb = std::min(std::max(1, rows / heads_wide), pow2_at_least(p.tokens));
    p.hb = rows / p.tb;
    // A block walks over all heads of its tokens unless that leaves multiprocessors without four blocks.
    const long long blocks_x = (p.tokens + (long long)p.tb - 1) / p.tb;
    const int rounds = (p.H + p.hb - 1) / p.hb;
    const long long want = 4LL * n_sm;
    const int split = (int)std::min<long long>(rounds, std::max<long long>(1, (want + blocks_x - 1) / blocks_x));
    p.heads_block = (rounds + split - 1) / split * p.hb;
    const dim3 grid((unsigned)blocks_x, (unsigned)((p.H + p.heads_block - 1) / p.heads_block));
    const bool staged = !t.interleaved && t.rot % 16 != 0;
    const size_t smem = staged ? (size_t)rows * (d * (f32 ? 4 : 2) + 4) : 0;
    auto go = [&](auto* f) { return launch_dependent(f, grid, kThreads, (int)smem, stream, p); };
    if (staged) return f32 ? go(rope_kernel<float, true, true, 1>) : go(rope_kernel<__nv_bfloat16, true, true, 1>);
    if (t.interleaved)
        return f32 ? go(rope_kernel<float, false, false, 2>) : go(rope_kernel<__nv_bfloat16, false, false, 2>);
    return f32 ? go(rope_kernel<float, true, false, 2>) : go(rope_kernel<__nv_bfloat16, true, false, 2>);
}

}  // namespace attn
