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
    bool e4m3 = false;
    int box_rows = 16;
    int device = 0, n_sm = 0;
};

namespace attn {

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
