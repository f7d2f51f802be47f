// Rotary positions: what the host hands to the kernels, and the device parts they share.
//
// Pair p of a head turns by the angle f_p * position.  The angle is kept as a fraction of a turn in 64-bit
// fixed point: step[p] = f_p / (2 pi) * 2^64, so position * step[p] modulo 2^64 is the phase with all whole turns
// gone, and without a rounding of its own.  What it is off by is position times the step's error: f_p and its quotient
// are float64, f_p <= 1, and the roundings of the power, of a scaling, of pi and of the quotient come to less than 2^-53
// turns (2^-55 measured; the cut to an integer adds 2^-64), 7e-10 rad at position 2^20 and 1.5e-6 at 2^31.  A float32
// product f_p * position would be off by 2^-24 of the whole angle (0.06 rad at position 2^20 for p = 0), and float64 runs
// at a small fraction of the integer rate on this GPU.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace attn {

constexpr int kRopeMaxPairs = 128;

struct RopeTable {
    unsigned long long step[kRopeMaxPairs];
    float amp = 1.f;      // factor on the rotated elements
    int rot = 0;          // rotated elements of a head, the first ones (even)
    int interleaved = 0;  // pairs (2p, 2p + 1); otherwise (p, p + rot / 2)
};

struct RopeRows {  // rows of d contiguous elements; strides in elements
    const char* src = nullptr;
    char* dst = nullptr;
    long long sb = 0, sh = 0, ss = 0;  // src
    long long db = 0, dh = 0, ds = 0;  // dst
};

#ifdef __CUDACC__
// cos and sin of the phase of one pair.  The nearest quarter of a turn is taken off in integers, so that a float32 number
// of half turns holds the rest, an eighth of a turn at most, to 2^-27 (2.3e-8 rad; the cut to 32 bits adds 4e-10);
// sincospif is accurate to an ulp.  (The whole angle as one float32 number would be off by up to 9e-8 rad.)
__device__ __forceinline__ void rope_cos_sin(int position, unsigned long long step, float& c, float& s) {
    const unsigned long long phase = (unsigned long long)(long long)position * step;
    const unsigned quarter = ((unsigned)(phase >> 32) + 0x20000000u) >> 30;
    const int rest = (int)(unsigned)(phase >> 30);  // the bits below the quarters, as a signed number of 2^-33 half turns
    float c0, s0;
    sincospif((float)rest * 1.1641532182693481e-10f, &s0, &c0);
    c = quarter & 1 ? s0 : c0;
    s = quarter & 1 ? c0 : s0;
    c = __uint_as_float(__float_as_uint(c) ^ ((quarter + 1) << 30 & 0x80000000u));
    s = __uint_as_float(__float_as_uint(s) ^ (quarter << 30 & 0x80000000u));
}

// The 16 elements a lane holds, as two runs of 8 (a, b), and where the runs start in the row.  Lane u of the d / 16
// lanes of a row owns the pairs 8u .. 8u + 7, counted over the row as the rotated pairs first and then the elements
// that stay, two by two.  Interleaved pairs are then 16 neighbouring elements; pairs of halves are two runs of 8,
// which start on 8-element boundaries when rot is a multiple of 16 (other rot: rope_pair_index, element by element).
__device__ __forceinline__ void rope_runs(bool halves, int rot, int u, int& off_a, int& off_b) {
    const bool turned = halves && 16 * u < rot;
    off_a = turned ? 8 * u : 16 * u;
    off_b = turned ? rot / 2 + 8 * u : 16 * u + 8;
}
__device__ __forceinline__ void rope_pair_index(bool halves, int rot, int q, int& i0, int& i1) {
    const bool turned = halves && 2 * q < rot;
    i0 = turned ? q : 2 * q;
    i1 = turned ? q + rot / 2 : 2 * q + 1;
}
// How many of a lane's eight pairs are rotated (the first ones).  The others keep their elements: a turn by nothing would
// make a NaN of the partner of an infinity.
__device__ __forceinline__ int rope_live_pairs(int u, int rot) { return min(8, max(0, rot / 2 - 8 * u)); }
// Turns a lane's pairs: neighbours in x, or (HALVES) across its two runs x[0 .. 7] and x[8 .. 15], where `live` is 0 or 8.
// Pairs that are not rotated come with c = 1 and s = 0.
template <bool HALVES>
__device__ __forceinline__ void rope_turn(float (&x)[16], const float (&c)[8], const float (&s)[8], int live) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int i0 = HALVES ? e : 2 * e, i1 = HALVES ? 8 + e : 2 * e + 1;
        const bool on = live > (HALVES ? 0 : e);
        const float a = x[i0], b = x[i1];
        const float bs = on ? b * s[e] : 0.f, as = on ? a * s[e] : -0.f;
        x[i0] = a * c[e] - bs;
        x[i1] = b * c[e] + as;
    }
}
// Eight neighbouring elements as they are in memory, and as float.
template <class T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
    uint4 v;
};
template <>
struct Raw8<float> {
    float4 v, w;
};
__device__ __forceinline__ void fetch8(const __nv_bfloat16* p, Raw8<__nv_bfloat16>& r) {
    r.v = *reinterpret_cast<const uint4*>(p);
}
__device__ __forceinline__ void fetch8(const float* p, Raw8<float>& r) {
    r.v = reinterpret_cast<const float4*>(p)[0];
    r.w = reinterpret_cast<const float4*>(p)[1];
}
__device__ __forceinline__ void widen8(const Raw8<__nv_bfloat16>& r, float* x) {
    const uint4 v = r.v;
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void widen8(const Raw8<float>& r, float* x) {
    x[0] = r.v.x; x[1] = r.v.y; x[2] = r.v.z; x[3] = r.v.w;
    x[4] = r.w.x; x[5] = r.w.y; x[6] = r.w.z; x[7] = r.w.w;
}
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* x) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]), bf16_pair(x[4], x[5]), bf16_pair(x[6], x[7]));
}
__device__ __forceinline__ void store8(float* p, const float* x) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
// The lane's cosines and sines from a table of its token's pairs, times amp.
__device__ __forceinline__ void rope_lane_turns(const float2* table, int u, int rot, float (&c)[8], float (&s)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int q = 8 * u + e;
        const float2 t = 2 * q < rot ? table[q] : make_float2(1.f, 0.f);  // (the table ends there)
        c[e] = t.x;
        s[e] = t.y;
    }
}
#endif

}  // namespace attn
