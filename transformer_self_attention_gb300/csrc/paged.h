// Launch parameters of the rotary, paged-cache and paged-decode kernels, and the arithmetic that host and device
// share: how the paged decode work is cut over the grid.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "attn.h"
#include "rope.h"

namespace attn {

// One launch for the rows of Q and K (Hk = 0: Q alone).
cudaError_t launch_rope(const RopeTable& t, const RopeRows& q, const RopeRows& k, int Hq, int Hk, int B, int S, int d,
                        const int* positions, long long pos_b, long long pos_s, bool inverse, bool f32, int n_sm,
                        cudaStream_t stream);

// ---------------------------------------------------------------- cache
// Bits of a cache's device error word.
constexpr int kCacheErrPosition = 1;  // a length or a row's position lies outside the page table
constexpr int kCacheErrPage = 2;      // a page number outside [0, n_pages)
constexpr int kCacheErrWait = 4;      // a bounded wait of the decode kernel ran out

// Layout: pages [n_pages, Hkv, 2, page, d] (keys, then values), bf16 or E4M3; scales (E4M3)
// [n_pages, Hkv, page / 16, 2, 16], the biased exponent e of each row's factor 2^(e - 127), 255 for a row
// that held an infinity or a NaN.  One 32-byte block of scales belongs to 16 positions of one kv head.
struct CacheView {
    char* pages = nullptr;
    uint8_t* scales = nullptr;
    int n_pages = 0, Hkv = 0, page = 0, d = 0;
    int* err = nullptr;
};
struct PageTable {
    const int* pages = nullptr;  // [B, max_pages], row stride `stride`
    const int* len = nullptr;    // [B]
    long long stride = 0;
    int max_pages = 0;
};
struct CacheWriteParams {
    CacheView c;
    PageTable t;
    RopeTable rope;       // rot = 0: K and Q are taken as they are
    RopeRows q, k, v;     // dst of k and v unused
    const int* new_len;   // [B], or null: S rows of every sequence
    int Hq, B, S;
};
struct CacheReadParams {
    CacheView c;
    PageTable t;
    RopeRows k, v;  // src unused
    int B, S, first;
};
cudaError_t launch_cache_write(const CacheWriteParams& p, bool e4m3, int n_sm, cudaStream_t stream);
cudaError_t launch_cache_read(const CacheReadParams& p, bool e4m3, cudaStream_t stream);

// ---------------------------------------------------------------- paged decode
// Work units are (sequence, kv head), in that order (over E4M3 pages with more than 32 rows to a head, (sequence, kv head,
// half of the rows): the second half finds its keys and values in L2).  A unit of n key blocks costs max(n, least) +
// overhead: its start, its merge and its output cost about as much as `overhead` blocks, and a unit of few blocks is not
// worth cutting (joining its parts costs more than the other blocks' time), so that units up to `least` all cost the same
// and the cuts fall between them.  Sequences without keys cost nothing.  The cost line [0, W) is cut into C intervals, equal
// but for one, one per CTA.  Inside a unit the blocks follow the overhead; a CTA takes the blocks whose cost positions
// its interval covers.
// Measured, bf16 (blocks of 8 KB): overheads of 10, 16, 22 and 30 blocks give 28.1, 27.1, 26.7 and 27.8 us for 16 ragged
// multi-query sequences of up to 16K positions and 169, 167, 168 and 169 us for 256 of up to 2K; least of 8, 12, 16 and
// 24 give 9.3, 9.7, 5.8 and 5.8 us for one sequence of 256 positions and 10.8, 11.0, 11.1 and 12.4 for one of 4K.  E4M3
// (tiles of 32 KB): overheads of 2, 3, 4 and 6 tiles give 27.9, 27.6, 27.7 and 28.1 us for 8 sequences of 1K to 8K, and
// least of 1, 2, 3 and 4 give 9.6, 6.8, 6.9 and 6.9 us, and 11.7, 12.9, 14.4 and 14.6, for the two sequences above.
struct PagedShape {
    int keys;  // positions of a key block
    unsigned overhead, least;
};
__host__ __device__ constexpr PagedShape paged_shape(int d, bool e4m3) {
    return e4m3 ? PagedShape{128, 3, 2} : PagedShape{d == 64 ? 32 : 16, 16, 16};
}
constexpr int kPagedMaxBatch = ATTN_DECODE_MAX_BATCH;
constexpr int kPagedMostPositions = 1 << 30;  // of a sequence; windows are cut to it

// Key blocks [lo, hi) of `keys` positions that some row of a sequence of length n can see.
__host__ __device__ inline void paged_blocks(int n, int S_q, int window, int keys, int& lo, int& hi) {
    hi = (n + keys - 1) / keys;
    const int first = window < 0 ? 0 : n - S_q - window;
    lo = first > 0 ? first / keys : 0;
}
__host__ __device__ inline unsigned paged_cost(int n, PagedShape s) {
    return n == 0 ? 0 : ((unsigned)n < s.least ? s.least : (unsigned)n) + s.overhead;
}
struct PagedCuts {
    unsigned C, q, r;  // CTAs; the intervals cost q + 1 for the first r, q for the others
    // One CTA per unit, more where the intervals still cost as much as a short unit.
    __host__ __device__ PagedCuts(unsigned W, unsigned units, unsigned grid, PagedShape s) {
        C = W / (s.least + s.overhead);
        C = C < units ? units : C;
        C = C < grid ? C : grid;
        C = C < 1 ? 1 : C;
        q = W / C;
        r = W - q * C;
    }
    __host__ __device__ unsigned begin(unsigned c) const { return c * q + (c < r ? c : r); }
    __host__ __device__ unsigned owner(unsigned x) const {  // the CTA whose interval holds cost position x
        const unsigned wide = r * (q + 1);
        return x < wide ? x / (q + 1) : r + (x - wide) / q;
    }
};
// Whether a launch may cut a unit at all, for any lengths up to `room` positions.
__host__ __device__ inline bool paged_may_cut(long long units, long long room, int grid, PagedShape s) {
    return units > grid || room > (long long)s.least * s.keys;
}

struct PagedParams {
    CUtensorMap tm;  // the pages, one box: 16 positions' keys and values (bf16), or box_rows keys or values (E4M3)
    const void* q;   // [B, Hq, S_q, d] bf16
    void* o;
    float* lse;      // may be null
    CacheView c;
    PageTable t;
    float* part_o;        // [2 * grid][rows_pad][d] unscaled sums, two slots per CTA: its first and its last stretch
    float2* part_ml;      // [2 * grid][rows_pad]: the rows' reference (base 2) and sum
    // Where the joining kernel finds the cut units.  By unit, where there are no more of them than CTAs: the first and the
    // last CTA that hold parts of it; otherwise by CTA: the unit that begins in it and ends in a later one, and that one.
    // x = -1: none.
    int2* cut;
    int by_unit;
    int B, Hq, Hkv, S_q, rows;
    int units;            // of a sequence: Hkv, times 2 where a head's rows are taken in two blocks
    int window;           // -1: none
    int causal;           // 0: every row sees every cached position
    int box_rows;         // E4M3: positions of a TMA box, a divisor of the page size
    float scale_log2;
    long long watchdog_ns;
    int withhold;  // test hook: a loading warp stops in front of the withhold-th key block of a batch (0: never)
};
// Rows a slot of the partial results is padded to, the blocks that a kv head's rows are taken in, and the CTAs of a full
// grid per multiprocessor.
int paged_rows_pad(int rows, bool e4m3);
int paged_row_blocks(int rows, bool e4m3);
int paged_ctas_per_sm(int rows, bool e4m3);
constexpr int kPagedMostCtasPerSm = 2;
cudaError_t launch_paged_bf16(const PagedParams& p, int grid, cudaStream_t stream);
cudaError_t launch_paged_e4m3(const PagedParams& p, int grid, cudaStream_t stream);
// Joins the parts of cut units; enqueued behind either as a programmatic dependent.
cudaError_t launch_paged_merge(const PagedParams& p, int grid, int rows_pad, cudaStream_t stream);

}  // namespace attn
