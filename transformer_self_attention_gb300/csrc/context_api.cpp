// Host implementation of the entry points of include/attn.h for long contexts over a paged cache: page bounds and
// selection, attention weights and eviction, shared prefixes.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>
#include <utility>

#include "attn.h"
#include "paged.h"
#include "paged_host.h"

struct attn_prefix_plan {
    attn_paged_plan* step = nullptr;  // of the own positions
    attn::OwnParts own;
    float* part_o = nullptr;
    float2* part_ml = nullptr;
    int4* groups = nullptr;
    int2* place = nullptr;
};

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

// Whether `count` ints at p share memory with a row of an int array: `rows` rows of `width`, `stride` ints apart.
bool meets(const int* p, long long count, const int* array, long long rows, long long width, long long stride) {
    if (!array) return false;
    const long long lo = ((long long)reinterpret_cast<uintptr_t>(p) - (long long)reinterpret_cast<uintptr_t>(array)) / 4;
    const long long hi = lo + count;  // (both are aligned) row r holds [r stride, r stride + width)
    if (stride == 0 || rows == 1) return lo < width && hi > 0;
    const long long last = hi <= 0 ? -1 : std::min(rows - 1, (hi - 1) / stride);  // the last row that begins in front of hi
    return last >= 0 && last * stride + width > lo;
}

attn_status done(cudaError_t e) { return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA; }

}  // namespace

extern "C" {

attn_status attn_bounds_update(attn_cache_handle h, void* codes, void* exponents, int B, const int* page_table,
                               long long table_stride, int max_pages, const int* cache_len, const int* new_len,
                               void* stream) {
    if (!h || !codes || !aligned(codes, 16) || !exponents || B < 1) return ATTN_ERR_INVALID_ARG;
    if (!table_ok(page_table, table_stride, max_pages, cache_len) || !aligned(new_len, 4)) return ATTN_ERR_INVALID_ARG;
    // (changed pages and heads are counted in 31 bits)
    if (B > ATTN_DECODE_MAX_BATCH || !room_ok(h, max_pages) || (long long)B * max_pages > 0x7FFFFFFFLL / h->c.Hkv)
        return ATTN_ERR_UNSUPPORTED;
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
    if (!out_table || !aligned(out_table, 4) || !out_len || !aligned(out_len, 4)) return ATTN_ERR_INVALID_ARG;
    const attn_status vs = attn::validate_paged(B, Hq, h->c.Hkv, S_q, ATTN_MASK_CAUSAL, 0);
    if (vs != ATTN_OK) return vs;
    // the new rows' own positions lie in the latest pages
    if (sinks < 0 || recent < 1 || recent - 1 < (S_q - 1 + h->c.page - 1) / h->c.page || (long long)sinks + recent > keep)
        return ATTN_ERR_INVALID_ARG;
    if (max_pages > attn::kSelectMostPages || keep > attn::kSelectMostPages || !room_ok(h, max_pages) ||
        (long long)B * h->c.Hkv > (1LL << 24))
        return ATTN_ERR_UNSUPPORTED;
    const long long places = (long long)B * h->c.Hkv * keep;
    if (meets(out_len, B, out_table, 1, places, 0)) return ATTN_ERR_INVALID_ARG;
    for (const auto& [out, count] : {std::pair{out_table, places}, std::pair{out_len, (long long)B}})
        if (meets(out, count, page_table, B, max_pages, table_stride) || meets(out, count, cache_len, 1, B, 0))
            return ATTN_ERR_INVALID_ARG;
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
    if (!h || !weights || !aligned(weights, 16) || !Q || !aligned(Q, 16) || !LSE || !aligned(LSE, 4))
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
    p.g.tm = h->keys_map;
    p.g.watchdog_ns = 2000000000LL;
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
    if (!h || !weights || !aligned(weights, 16) || B < 1) return ATTN_ERR_INVALID_ARG;
    if (!table_ok(page_table, table_stride, max_pages, cache_len)) return ATTN_ERR_INVALID_ARG;
    if (keep < 0 || recent < 0 || (long long)keep + recent < 1 || !out_len || !aligned(out_len, 4) || !kept ||
        !aligned(kept, 4))
        return ATTN_ERR_INVALID_ARG;
    const long long stay = (long long)keep + recent, room = (long long)max_pages * h->c.page;
    if (to_table) {
        if (!table_ok(to_table, to_stride, to_max_pages, cache_len) || to_table == page_table ||
            (long long)to_max_pages * h->c.page < std::min(stay, room))
            return ATTN_ERR_INVALID_ARG;
    }
    if (B > ATTN_DECODE_MAX_BATCH || !room_ok(h, max_pages) || stay > attn::kPagedMostPositions ||
        (long long)B * h->c.Hkv * ((std::min(stay, room) + 7) / 8) > (1LL << 30))
        return ATTN_ERR_UNSUPPORTED;
    const long long places = (long long)B * h->c.Hkv * stay;
    if (meets(out_len, B, kept, 1, places, 0)) return ATTN_ERR_INVALID_ARG;
    for (const auto& [out, count] : {std::pair{kept, places}, std::pair{out_len, (long long)B}})
        if (meets(out, count, page_table, B, max_pages, table_stride) || meets(out, count, cache_len, 1, B, 0) ||
            meets(out, count, to_table, B, to_max_pages, to_stride))
            return ATTN_ERR_INVALID_ARG;
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
    return done(attn::launch_evict(p, h->e4m3, h->n_sm, static_cast<cudaStream_t>(stream)));
}

attn_status attn_prefix_create(attn_prefix_handle* out, int B, int Hq, int Hkv, int S_q, int d, float scale,
                               attn_mask_kind kind) {
    if (!out) return ATTN_ERR_INVALID_ARG;
    *out = nullptr;
    if (kind != ATTN_MASK_FULL && kind != ATTN_MASK_CAUSAL)
        return (int)kind < ATTN_MASK_FULL || (int)kind > ATTN_MASK_LOCAL_GLOBAL ? ATTN_ERR_INVALID_ARG : ATTN_ERR_UNSUPPORTED;
    attn_prefix_plan* h = new (std::nothrow) attn_prefix_plan();
    if (!h) return ATTN_ERR_OOM;
    attn_status st = attn_paged_create(&h->step, B, Hq, Hkv, S_q, d, scale, kind, 0);
    if (st != ATTN_OK) {
        delete h;
        return st;
    }
    const size_t rows = (size_t)B * Hq * S_q;
    const size_t parts = 2 * (rows + (size_t)attn::kPrefixTile * h->step->n_sm);
    auto get = [&](auto& p, size_t n) {
        if (st != ATTN_OK) return;
        const cudaError_t e = cudaMalloc(reinterpret_cast<void**>(&p), n * sizeof(*p));
        if (e != cudaSuccess) st = e == cudaErrorMemoryAllocation ? ATTN_ERR_OOM : ATTN_ERR_CUDA;
    };
    get(h->own.whole_o, rows * d);
    get(h->own.whole_ml, rows);
    get(h->own.cut, (size_t)B * Hkv * 2);
    get(h->part_o, parts * d);
    get(h->part_ml, parts);
    get(h->groups, ATTN_DECODE_MAX_BATCH + 1);
    get(h->place, B);
    if (st != ATTN_OK) {
        attn_prefix_destroy(h);
        return st;
    }
    *out = h;
    return ATTN_OK;
}

attn_status attn_prefix_forward(attn_prefix_handle h, attn_cache_handle cache, const void* Q, const int* prefix_table,
                                long long prefix_stride, int prefix_max_pages, const int* prefix_len, int n_prefix,
                                const int* prefix_of, const int* page_table, long long table_stride, int max_pages,
                                const int* cache_len, void* O, float* LSE, void* stream) {
    if (!h || !cache) return ATTN_ERR_INVALID_ARG;
    if (!table_ok(prefix_table, prefix_stride, prefix_max_pages, prefix_len) || n_prefix < 1 || !aligned(prefix_of, 4) ||
        (!prefix_of && n_prefix != 1))
        return ATTN_ERR_INVALID_ARG;
    if (!table_ok(page_table, table_stride, max_pages, cache_len) || !Q || !aligned(Q, 16) || !O || !aligned(O, 16) ||
        !aligned(LSE, 4))
        return ATTN_ERR_INVALID_ARG;
    attn_paged_plan* s = h->step;
    if (cache->c.Hkv != s->Hkv || cache->c.d != s->d || cache->device != s->device || !on_device(s->device))
        return ATTN_ERR_INVALID_ARG;
    const int rows = s->Hq / s->Hkv * s->S_q;
    if (n_prefix > ATTN_DECODE_MAX_BATCH || !room_ok(cache, prefix_max_pages) || !room_ok(cache, max_pages))
        return ATTN_ERR_UNSUPPORTED;
    // the line of cost fits an int: every unit, and every prefix's last one
    const long long tiles = (long long)prefix_max_pages * cache->c.page / attn::kPrefixTile + 8;
    if (2 * tiles * s->Hkv * ((long long)n_prefix + (long long)s->B * rows / attn::kPrefixTile) > 0x7FFFFFFFLL)
        return ATTN_ERR_UNSUPPORTED;
    attn::PrefixParams p{};
    p.tm = cache->e4m3 ? cache->map : cache->rows_map;
    p.c = cache->c;
    p.t = table_of(prefix_table, prefix_stride, prefix_max_pages, prefix_len);
    p.of = prefix_of;
    p.q = Q;
    p.B = s->B; p.G = n_prefix; p.Hkv = s->Hkv; p.rows = rows;
    p.box_rows = cache->box_rows;
    p.part_o = h->part_o; p.part_ml = h->part_ml; p.groups = h->groups; p.place = h->place;
    p.scale_log2 = (float)((double)s->scale * 1.4426950408889634);
    p.watchdog_ns = s->watchdog_ns;
    p.withhold = s->withhold;
    const int grid = std::min(s->n_sm, s->grid_limit);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (attn::launch_prefix(p, cache->e4m3, grid, st) != cudaSuccess) return ATTN_ERR_CUDA;
    attn::OwnParts own = h->own;
    const attn_status r = attn::paged_step(s, cache, Q, page_table, table_stride, 0, max_pages, cache_len, O, LSE, &own, stream);
    if (r != ATTN_OK) return r;
    attn::JoinParams j{};
    j.whole_o = own.whole_o; j.whole_ml = own.whole_ml;
    j.part_o = s->d_part; j.part_ml = s->d_ml; j.cut = own.cut;
    j.rows_pad = own.rows_pad; j.row_blocks = own.row_blocks;
    j.o = O; j.lse = LSE;
    return done(attn::launch_join(p, j, st));
}

attn_status attn_prefix_set_grid_limit(attn_prefix_handle h, int max_ctas) {
    return h ? attn_paged_set_grid_limit(h->step, max_ctas) : ATTN_ERR_INVALID_ARG;
}

attn_status attn_prefix_set_watchdog(attn_prefix_handle h, long long limit_ns, int withhold) {
    return h ? attn_paged_set_watchdog(h->step, limit_ns, withhold) : ATTN_ERR_INVALID_ARG;
}

attn_status attn_prefix_destroy(attn_prefix_handle h) {
    if (!h) return ATTN_OK;
    const attn_status st = attn_paged_destroy(h->step);  // (synchronises the device)
    for (void* p : {(void*)h->own.whole_o, (void*)h->own.whole_ml, (void*)h->own.cut, (void*)h->part_o, (void*)h->part_ml,
                    (void*)h->groups, (void*)h->place})
        if (p) cudaFree(p);
    delete h;
    return st;
}

}  // extern "C"
