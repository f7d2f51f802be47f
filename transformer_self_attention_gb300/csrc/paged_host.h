// Host side that the entry points over a paged cache share: the handles, and the checks of their arguments.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "attn.h"
#include "device_once.h"
#include "paged.h"

struct attn_rope_plan {
    attn::RopeTable t;
    double freq[attn::kRopeMaxPairs] = {};
    double amplitude = 1.0;
    int d = 0;
};

struct attn_cache_plan {
    attn::CacheView c;
    CUtensorMap map{};
    CUtensorMap keys_map{};  // the keys of 16 positions
    CUtensorMap rows_map{};  // bf16: boxes of box_rows positions, 128 bytes of their keys or values
    bool e4m3 = false;
    int box_rows = 16;
    int device = 0, n_sm = 0;
};

struct attn_paged_plan {
    int B = 0, Hq = 0, Hkv = 0, S_q = 0, d = 0, kind = 0, window = 0;
    int device = 0, n_sm = 0;
    int grid_limit = 1 << 30;
    long long watchdog_ns = 2000000000LL;
    int withhold = 0;
    float scale = 0.f;
    float* d_part = nullptr;
    float2* d_ml = nullptr;
    int2* d_cut = nullptr;
};

namespace attn {

// A decode step that leaves its parts to be joined by somebody else: where they go (cut: [B * units], by unit), and, filled
// in by the step, how they lie there.
struct OwnParts {
    float* whole_o = nullptr;
    float2* whole_ml = nullptr;
    int2* cut = nullptr;
    int rows_pad = 0, row_blocks = 0;
};
// attn_paged_forward_heads, or with `own` the part of it before the joining of cut units.
attn_status paged_step(attn_paged_plan* h, attn_cache_plan* cache, const void* Q, const int* page_table,
                       long long table_stride, long long head_stride, int max_pages, const int* cache_len, void* O,
                       float* LSE, OwnParts* own, void* stream);

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

inline bool on_device(int device) {
    int dev = -1;
    return cudaGetDevice(&dev) == cudaSuccess && dev == device;
}

inline bool table_ok(const int* page_table, long long stride, int max_pages, const int* cache_len) {
    return page_table && aligned(page_table, 4) && cache_len && aligned(cache_len, 4) && max_pages >= 1 &&
           max_pages <= (1 << 26) && stride >= 0;
}

inline attn_status validate_paged(int B, int Hq, int Hkv, int S_q, attn_mask_kind kind, int window) {
    if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || S_q < 1) return ATTN_ERR_INVALID_ARG;
    if ((int)kind < ATTN_MASK_FULL || (int)kind > ATTN_MASK_LOCAL_GLOBAL) return ATTN_ERR_INVALID_ARG;
    if (kind != ATTN_MASK_FULL && kind != ATTN_MASK_CAUSAL && kind != ATTN_MASK_CAUSAL_SLIDING)
        return ATTN_ERR_UNSUPPORTED;
    if (kind == ATTN_MASK_CAUSAL_SLIDING && window < 0) return ATTN_ERR_INVALID_ARG;
    if (B > ATTN_DECODE_MAX_BATCH || (long)(Hq / Hkv) * S_q > ATTN_DECODE_MAX_ROWS || Hkv > (1 << 16))
        return ATTN_ERR_UNSUPPORTED;
    return ATTN_OK;
}

// A window of 2^30 sees every position there can be; with more, a difference of positions would pass 32 bits.
inline int window_of(attn_mask_kind kind, int window) {
    return kind == ATTN_MASK_CAUSAL_SLIDING ? std::min(window, attn::kPagedMostPositions) : -1;
}

}  // namespace attn
