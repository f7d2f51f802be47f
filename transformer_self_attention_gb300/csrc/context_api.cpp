// Host implementation of the entry points of include/attn.h for long contexts over a paged cache: page bounds and selection.
#include <cuda_runtime.h>

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

}  // extern "C"
