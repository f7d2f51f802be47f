// Host implementation of the entry points of include/attn.h for long contexts over a paged cache: page bounds and
// selection, attention weights and eviction.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "attn.h"
#include "paged.h"
#include "paged_host.h"

using attn::aligned;
using attn::on_device;
using attn::table_ok;

namespace {

attn::PageTable table_of(const int* page_table, long long stride, int max_pages, const int* cache_len) {
    attn::PageTable t;
    t.pages = page_table;
    t.len = cache_len;
    t.stride = stride;
    t.max_pages = max_pages;
    return t;
}
// Positions of a row of the table fit an int with room for differences.
bool room_ok(attn_cache_handle h, int max_pages) { return (long long)max_pages * h->c.page <= attn::kPagedMostPositions; }

attn_status done(cudaError_t e) { return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA; }

}  // namespace

extern "C" {

attn_status attn_bounds_update(attn_cache_handle h, void* codes, void* exponents, int B, const int* page_table,
                               long long table_stride, int max_pages, const int* cache_len, const int* new_len,
                               void* stream) {
    if (!h || !codes || !aligned(codes, 16) || !exponents || B < 1) return ATTN_ERR_INVALID_ARG;
    if (!table_ok(page_table, table_stride, max_pages, cache_len) || !aligned(new_len, 4)) return ATTN_ERR_INVALID_ARG;
    if (B > ATTN_DECODE_MAX_BATCH || !room_ok(h, max_pages)) return ATTN_ERR_UNSUPPORTED;
    if (!on_device(h->device)) return ATTN_ERR_INVALID_ARG;
    attn::BoundsParams p{};
    p.c = h->c;
    p.t = table_of(page_table, table_stride, max_pages, cache_len);
    p.codes = static_cast<int8_t*>(codes);
    p.exps = static_cast<uint8_t*>(exponents);
    p.new_len = new_len;
    p.B = B;
    return done(attn::launch_bounds_update(p, h->e4m3, h->n_sm, static_cast<cudaStream_t>(stream)));
}

attn_status attn_bounds_select(attn_cache_handle h, const void* codes, const void* exponents, int B, int Hq, int S_q,
                               const void* Q, const int* page_table, long long table_stride, int max_pages,
                               const int* cache_len, int keep, int sinks, int recent, int* out_table, int* out_len,
                               void* stream) {
    if (!h || !codes || !aligned(codes, 16) || !exponents || !Q || !aligned(Q, 16)) return ATTN_ERR_INVALID_ARG;
    if (!table_ok(page_table, table_stride, max_pages, cache_len)) return ATTN_ERR_INVALID_ARG;
    if (!out_table || !aligned(out_table, 4) || out_table == page_table || !out_len || !aligned(out_len, 4) ||
        out_len == cache_len)
        return ATTN_ERR_INVALID_ARG;
    const attn_status vs = attn::validate_paged(B, Hq, h->c.Hkv, S_q, ATTN_MASK_CAUSAL, 0);
    if (vs != ATTN_OK) return vs;
    // the new rows' own positions lie in the latest pages
    if (sinks < 0 || recent < 1 || recent - 1 < (S_q - 1 + h->c.page - 1) / h->c.page || (long long)sinks + recent > keep)
        return ATTN_ERR_INVALID_ARG;
    if (max_pages > attn::kSelectMostPages || keep > attn::kSelectMostPages || !room_ok(h, max_pages) ||
        (long long)B * h->c.Hkv > (1LL << 24))
        return ATTN_ERR_UNSUPPORTED;
    if (!on_device(h->device)) return ATTN_ERR_INVALID_ARG;
    attn::SelectParams p{};
    p.c = h->c;
    p.t = table_of(page_table, table_stride, max_pages, cache_len);
    p.codes = static_cast<const int8_t*>(codes);
    p.exps = static_cast<const uint8_t*>(exponents);
    p.q = Q;
    p.B = B; p.Hkv = h->c.Hkv; p.rows = Hq / h->c.Hkv * S_q;
    p.keep = keep; p.sinks = sinks; p.recent = recent;
    p.out_table = out_table;
    p.out_len = out_len;
    return done(attn::launch_bounds_select(p, h->n_sm, static_cast<cudaStream_t>(stream)));
}

attn_status attn_weights_accumulate(attn_cache_handle h, float* weights, int B, int Hq, int S_q, const void* Q,
                                    const float* LSE, float scale, attn_mask_kind kind, int window, float decay,
                                    const int* page_table, long long table_stride, int max_pages, const int* cache_len,
                                    void* stream) {
    if (!h || !weights || !aligned(weights, 4) || !Q || !aligned(Q, 16) || !LSE || !aligned(LSE, 4))
        return ATTN_ERR_INVALID_ARG;
    if (!table_ok(page_table, table_stride, max_pages, cache_len)) return ATTN_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || !(scale > 0.f) || !(decay >= 0.f && decay <= 1.f)) return ATTN_ERR_INVALID_ARG;
    const attn_status vs = attn::validate_paged(B, Hq, h->c.Hkv, S_q, kind, window);
    if (vs != ATTN_OK) return vs;
    // a sequence's cost, and all of them, fit the split's numbers
    const long long most = 64 + (long long)max_pages * h->c.page / 16;
    if (!room_ok(h, max_pages) || most * B * h->c.Hkv > 0x7FFFFFFFLL) return ATTN_ERR_UNSUPPORTED;
    if (!on_device(h->device)) return ATTN_ERR_INVALID_ARG;
    attn::WeighParams p{};
    p.g.q = Q;
    p.g.c = h->c;
    p.g.t = table_of(page_table, table_stride, max_pages, cache_len);
    p.g.B = B; p.g.Hq = Hq; p.g.Hkv = p.g.units = h->c.Hkv; p.g.S_q = S_q;
    p.g.rows = Hq / h->c.Hkv * S_q;
    p.g.causal = kind != ATTN_MASK_FULL;
    p.g.scale_log2 = (float)((double)scale * 1.4426950408889634);
    p.window = attn::window_of(kind, window);
    p.g.window = decay == 1.f ? p.window : -1;  // positions before the window fade too
    p.lse = LSE;
    p.w = weights;
    p.decay = decay;
    return done(attn::launch_weigh(p, h->e4m3, h->n_sm, static_cast<cudaStream_t>(stream)));
}

attn_status attn_weights_evict(attn_cache_handle h, float* weights, int B, const int* page_table, long long table_stride,
                               int max_pages, const int* cache_len, int keep, int recent, const int* to_table,
                               long long to_stride, int to_max_pages, int* out_len, int* kept, void* stream) {
    if (!h || !weights || !aligned(weights, 4) || B < 1) return ATTN_ERR_INVALID_ARG;
    if (!table_ok(page_table, table_stride, max_pages, cache_len)) return ATTN_ERR_INVALID_ARG;
    if (keep < 0 || recent < 0 || (long long)keep + recent < 1 || !out_len || !aligned(out_len, 4) || !kept ||
        !aligned(kept, 4) || out_len == cache_len || kept == page_table)
        return ATTN_ERR_INVALID_ARG;
    const long long stay = (long long)keep + recent, room = (long long)max_pages * h->c.page;
    if (to_table) {
        if (!table_ok(to_table, to_stride, to_max_pages, cache_len) || to_table == page_table || kept == to_table ||
            (long long)to_max_pages * h->c.page < std::min(stay, room))
            return ATTN_ERR_INVALID_ARG;
    }
    if (B > ATTN_DECODE_MAX_BATCH || !room_ok(h, max_pages) || stay > attn::kPagedMostPositions ||
        (long long)B * h->c.Hkv * ((std::min(stay, room) + 31) / 32) > 0x7FFFFFFFLL)
        return ATTN_ERR_UNSUPPORTED;
    if (!on_device(h->device)) return ATTN_ERR_INVALID_ARG;
    attn::EvictParams p{};
    p.c = h->c;
    p.t = table_of(page_table, table_stride, max_pages, cache_len);
    p.w = weights;
    p.to = to_table;
    p.to_stride = to_stride;
    p.out_len = out_len;
    p.kept = kept;
    p.B = B; p.keep = keep; p.recent = recent;
    p.in_place = !to_table;
    return done(attn::launch_evict(p, h->e4m3, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
