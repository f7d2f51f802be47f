// Host implementation of the rotary, paged-cache and paged-decode entry points of include/attn.h.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>
#include <new>
#include <vector>

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

namespace {

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    });
    return fn;
}

// bf16 pages as {row part, slots, parts of a row, K / V, page * Hkv + head}: a row comes in parts of 128 bytes, one box
// holds 16 positions' keys and values of one head.
bool encode_bf16(CUtensorMap* map, const attn::CacheView& c) {
    auto enc = encoder();
    if (!enc) return false;
    const int row = c.d * 2, parts = row / 128;
    cuuint64_t dims[5] = {64, (cuuint64_t)c.page, (cuuint64_t)parts, 2, (cuuint64_t)c.n_pages * c.Hkv};
    cuuint64_t strides[4] = {(cuuint64_t)row, 128, (cuuint64_t)c.page * row, (cuuint64_t)2 * c.page * row};
    cuuint32_t box[5] = {64, 16, (cuuint32_t)parts, 2, 1};
    cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, c.pages, dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// E4M3 pages as {row, slots, K / V, page * Hkv + head}; one box holds `rows` positions' keys or values of one head.
bool encode_e4m3(CUtensorMap* map, const attn::CacheView& c, int rows) {
    auto enc = encoder();
    if (!enc) return false;
    cuuint64_t dims[4] = {(cuuint64_t)c.d, (cuuint64_t)c.page, 2, (cuuint64_t)c.n_pages * c.Hkv};
    cuuint64_t strides[3] = {(cuuint64_t)c.d, (cuuint64_t)c.page * c.d, (cuuint64_t)2 * c.page * c.d};
    cuuint32_t box[4] = {(cuuint32_t)c.d, (cuuint32_t)rows, 1, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, c.pages, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               c.d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Rows of `el`-byte elements: the first one and every stride on 16-byte boundaries.
bool rows_ok(const attn_rows* r, int el) {
    const long long unit = 16 / el;
    return r && r->data && aligned(r->data, 16) && r->stride_b % unit == 0 && r->stride_h % unit == 0 &&
           r->stride_s % unit == 0;
}
attn::RopeRows rows_of(const attn_rows* src, const attn_rows* dst) {
    attn::RopeRows r;
    if (src) {
        r.src = static_cast<const char*>(src->data);
        r.sb = src->stride_b; r.sh = src->stride_h; r.ss = src->stride_s;
    }
    if (dst) {
        r.dst = static_cast<char*>(dst->data);
        r.db = dst->stride_b; r.dh = dst->stride_h; r.ds = dst->stride_s;
    }
    return r;
}

// The error word set to zero, by the time the call returns: the caller's next launch may be on a stream that does not wait
// for the one this runs on, and what it records must not be wiped out.
bool clear_error(int* err) {
    return cudaMemset(err, 0, sizeof(int)) == cudaSuccess && cudaStreamSynchronize(cudaStreamLegacy) == cudaSuccess;
}

bool on_device(int device) {
    int dev = -1;
    return cudaGetDevice(&dev) == cudaSuccess && dev == device;
}

attn_status rope_apply(attn_rope_handle h, attn_dtype dtype, int B, int S, int Hq, const attn_rows* Q,
                       const attn_rows* Q_out, int Hk, const attn_rows* K, const attn_rows* K_out,
                       const int* positions, long long pos_stride_b, long long pos_stride_s, bool inverse,
                       void* stream) {
    if (!h || (dtype != ATTN_BF16 && dtype != ATTN_F32)) return ATTN_ERR_INVALID_ARG;
    if (B < 1 || S < 0 || Hq < 1 || Hk < 0 || Hq > (1 << 20) || Hk > (1 << 20)) return ATTN_ERR_INVALID_ARG;
    if (S == 0) return ATTN_OK;
    if ((long long)B * S > (1LL << 30)) return ATTN_ERR_UNSUPPORTED;
    const int el = dtype == ATTN_BF16 ? 2 : 4;
    if (!rows_ok(Q, el) || !rows_ok(Q_out, el)) return ATTN_ERR_INVALID_ARG;
    if (Hk > 0 && (!rows_ok(K, el) || !rows_ok(K_out, el))) return ATTN_ERR_INVALID_ARG;
    if (!aligned(positions, 4)) return ATTN_ERR_INVALID_ARG;
    const int n_sm = attn::current_sm_count();
    if (n_sm < 1) return ATTN_ERR_CUDA;
    const cudaError_t e = attn::launch_rope(h->t, rows_of(Q, Q_out), Hk > 0 ? rows_of(K, K_out) : attn::RopeRows{}, Hq,
                                            Hk, B, S, h->d, positions, pos_stride_b, pos_stride_s, inverse,
                                            dtype == ATTN_F32, n_sm, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

bool table_ok(const int* page_table, long long stride, int max_pages, const int* cache_len) {
    return page_table && aligned(page_table, 4) && cache_len && aligned(cache_len, 4) && max_pages >= 1 &&
           max_pages <= (1 << 26) && stride >= 0;
}

attn_status validate_paged(int B, int Hq, int Hkv, int S_q, attn_mask_kind kind, int window) {
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
int window_of(attn_mask_kind kind, int window) {
    return kind == ATTN_MASK_CAUSAL_SLIDING ? std::min(window, attn::kPagedMostPositions) : -1;
}

void free_paged(attn_paged_plan* h) {
    if (!h) return;
    if (h->d_part) cudaFree(h->d_part);
    if (h->d_ml) cudaFree(h->d_ml);
    if (h->d_cut) cudaFree(h->d_cut);
    delete h;
}

}  // namespace

extern "C" {

attn_status attn_rope_create(attn_rope_handle* out, int d, int rot, attn_rope_layout layout, double base,
                             attn_rope_scaling scaling, double factor, int original_len, double beta_fast,
                             double beta_slow, double amplitude) {
    if (!out) return ATTN_ERR_INVALID_ARG;
    *out = nullptr;
    if (rot < 2 || rot % 2 != 0 || rot > d) return ATTN_ERR_INVALID_ARG;
    if (layout != ATTN_ROPE_HALF && layout != ATTN_ROPE_INTERLEAVED) return ATTN_ERR_INVALID_ARG;
    if ((int)scaling < ATTN_ROPE_PLAIN || (int)scaling > ATTN_ROPE_YARN) return ATTN_ERR_INVALID_ARG;
    if (!std::isfinite(base) || !(base > 1.0) || !std::isfinite(amplitude) || amplitude < 0.0)
        return ATTN_ERR_INVALID_ARG;
    if (scaling != ATTN_ROPE_PLAIN && (!std::isfinite(factor) || !(factor >= 1.0))) return ATTN_ERR_INVALID_ARG;
    if (scaling == ATTN_ROPE_NTK && rot == 2) return ATTN_ERR_INVALID_ARG;
    if (scaling == ATTN_ROPE_YARN &&
        (original_len < 1 || !std::isfinite(beta_fast) || !std::isfinite(beta_slow) || !(beta_fast > beta_slow)))
        return ATTN_ERR_INVALID_ARG;
    if (d < 16 || d % 16 != 0 || d > 2 * attn::kRopeMaxPairs) return ATTN_ERR_UNSUPPORTED;
    attn_rope_plan* h = new (std::nothrow) attn_rope_plan();
    if (!h) return ATTN_ERR_OOM;
    const double pi = 3.14159265358979323846;
    const double b = scaling == ATTN_ROPE_NTK ? base * std::pow(factor, (double)rot / (rot - 2)) : base;
    for (int i = 0; i < rot / 2; ++i) {
        double f = std::pow(b, -2.0 * i / rot);
        if (scaling == ATTN_ROPE_LINEAR) f /= factor;
        if (scaling == ATTN_ROPE_YARN) {
            const double turns = original_len * f / (2.0 * pi);
            const double keep = std::min(1.0, std::max(0.0, (turns - beta_slow) / (beta_fast - beta_slow)));
            f = keep * f + (1.0 - keep) * f / factor;
        }
        h->freq[i] = f;
        // f <= 1, so f / (2 pi) < 1/4 of 2^64 turns' worth: no overflow
        h->t.step[i] = (unsigned long long)std::ldexp(f / (2.0 * pi), 64);
    }
    h->amplitude = amplitude > 0.0 ? amplitude : scaling == ATTN_ROPE_YARN ? 0.1 * std::log(factor) + 1.0 : 1.0;
    h->t.amp = (float)h->amplitude;
    h->t.rot = rot;
    h->t.interleaved = layout == ATTN_ROPE_INTERLEAVED;
    h->d = d;
    *out = h;
    return ATTN_OK;
}

attn_status attn_rope_frequencies(attn_rope_handle h, double* freq, double* amplitude) {
    if (!h || !freq || !amplitude) return ATTN_ERR_INVALID_ARG;
    for (int i = 0; i < h->t.rot / 2; ++i) freq[i] = h->freq[i];
    *amplitude = h->amplitude;
    return ATTN_OK;
}

attn_status attn_rope_forward(attn_rope_handle h, attn_dtype dtype, int B, int S, int Hq, const attn_rows* Q,
                              const attn_rows* Q_out, int Hk, const attn_rows* K, const attn_rows* K_out,
                              const int* positions, long long pos_stride_b, long long pos_stride_s, void* stream) {
    return rope_apply(h, dtype, B, S, Hq, Q, Q_out, Hk, K, K_out, positions, pos_stride_b, pos_stride_s, false,
                      stream);
}

attn_status attn_rope_backward(attn_rope_handle h, attn_dtype dtype, int B, int S, int Hq, const attn_rows* dQ_out,
                               const attn_rows* dQ, int Hk, const attn_rows* dK_out, const attn_rows* dK,
                               const int* positions, long long pos_stride_b, long long pos_stride_s, void* stream) {
    return rope_apply(h, dtype, B, S, Hq, dQ_out, dQ, Hk, dK_out, dK, positions, pos_stride_b, pos_stride_s, true,
                      stream);
}

attn_status attn_rope_destroy(attn_rope_handle h) {
    delete h;
    return ATTN_OK;
}

attn_status attn_cache_create(attn_cache_handle* out, int n_pages, int Hkv, int page, int d, attn_dtype dtype,
                              void* pages, void* scales) {
    if (!out) return ATTN_ERR_INVALID_ARG;
    *out = nullptr;
    if (n_pages < 1 || Hkv < 1 || page < 16 || page % 16 != 0 || !pages || !aligned(pages, 16))
        return ATTN_ERR_INVALID_ARG;
    if (dtype != ATTN_BF16 && dtype != ATTN_FP8_E4M3) return ATTN_ERR_UNSUPPORTED;
    if (dtype == ATTN_FP8_E4M3 && (!scales || !aligned(scales, 16))) return ATTN_ERR_INVALID_ARG;
    if ((d != 64 && d != 128) || page > 1024 || Hkv > (1 << 16) || (long long)n_pages * Hkv > (1LL << 31) - 1)
        return ATTN_ERR_UNSUPPORTED;
    attn_cache_plan* h = new (std::nothrow) attn_cache_plan();
    if (!h) return ATTN_ERR_OOM;
    h->e4m3 = dtype == ATTN_FP8_E4M3;
    h->c.pages = static_cast<char*>(pages);
    h->c.scales = h->e4m3 ? static_cast<uint8_t*>(scales) : nullptr;
    h->c.n_pages = n_pages; h->c.Hkv = Hkv; h->c.page = page; h->c.d = d;
    auto fail = [&](attn_status s) {
        if (h->c.err) cudaFree(h->c.err);
        delete h;
        return s;
    };
    if (cudaGetDevice(&h->device) != cudaSuccess || (h->n_sm = attn::current_sm_count()) < 1)
        return fail(ATTN_ERR_CUDA);
    const cudaError_t e = cudaMalloc(reinterpret_cast<void**>(&h->c.err), sizeof(int));
    if (e != cudaSuccess) return fail(e == cudaErrorMemoryAllocation ? ATTN_ERR_OOM : ATTN_ERR_CUDA);
    if (!clear_error(h->c.err)) return fail(ATTN_ERR_CUDA);
    // the largest power of two that divides the page, up to a decode tile
    while (h->box_rows < 128 && page % (2 * h->box_rows) == 0) h->box_rows *= 2;
    if (!(h->e4m3 ? encode_e4m3(&h->map, h->c, h->box_rows) : encode_bf16(&h->map, h->c))) return fail(ATTN_ERR_CUDA);
    *out = h;
    return ATTN_OK;
}

attn_status attn_cache_write(attn_cache_handle h, int B, int S_new, const attn_rows* K, const attn_rows* V,
                             const int* page_table, long long table_stride, int max_pages, const int* cache_len,
                             const int* new_len, attn_rope_handle rope, int Hq, const attn_rows* Q,
                             const attn_rows* Q_out, void* stream) {
    if (!h || B < 1 || S_new < 0 || Hq < 0 || Hq > (1 << 20)) return ATTN_ERR_INVALID_ARG;
    if (!table_ok(page_table, table_stride, max_pages, cache_len) || !aligned(new_len, 4)) return ATTN_ERR_INVALID_ARG;
    if (rope && rope->d != h->c.d) return ATTN_ERR_INVALID_ARG;
    if (S_new == 0) return ATTN_OK;  // (rows of nothing need no data)
    if (Hq > 0 && (!rows_ok(Q, 2) || !rows_ok(Q_out, 2))) return ATTN_ERR_INVALID_ARG;
    if (!rows_ok(K, 2) || !rows_ok(V, 2)) return ATTN_ERR_INVALID_ARG;
    if (B > ATTN_DECODE_MAX_BATCH || (long long)B * S_new > (1LL << 30)) return ATTN_ERR_UNSUPPORTED;
    if (!on_device(h->device)) return ATTN_ERR_INVALID_ARG;
    attn::CacheWriteParams p{};
    p.c = h->c;
    p.t.pages = page_table; p.t.len = cache_len; p.t.stride = table_stride; p.t.max_pages = max_pages;
    if (rope) p.rope = rope->t;
    p.q = Hq > 0 ? rows_of(Q, Q_out) : attn::RopeRows{};
    p.k = rows_of(K, nullptr);
    p.v = rows_of(V, nullptr);
    p.new_len = new_len;
    p.Hq = Hq; p.B = B; p.S = S_new;
    const cudaError_t e = attn::launch_cache_write(p, h->e4m3, h->n_sm, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

attn_status attn_cache_read(attn_cache_handle h, int B, int S, int first, const attn_rows* K, const attn_rows* V,
                            const int* page_table, long long table_stride, int max_pages, const int* cache_len,
                            void* stream) {
    if (!h || B < 1 || S < 0 || first < 0) return ATTN_ERR_INVALID_ARG;
    if (!table_ok(page_table, table_stride, max_pages, cache_len)) return ATTN_ERR_INVALID_ARG;
    if (S == 0) return ATTN_OK;
    if (!rows_ok(K, 2) || !rows_ok(V, 2)) return ATTN_ERR_INVALID_ARG;
    if (B > ATTN_DECODE_MAX_BATCH || S > (1 << 30)) return ATTN_ERR_UNSUPPORTED;
    if (!on_device(h->device)) return ATTN_ERR_INVALID_ARG;
    attn::CacheReadParams p{};
    p.c = h->c;
    p.t.pages = page_table; p.t.len = cache_len; p.t.stride = table_stride; p.t.max_pages = max_pages;
    p.k = rows_of(nullptr, K);
    p.v = rows_of(nullptr, V);
    p.B = B; p.S = S; p.first = first;
    const cudaError_t e = attn::launch_cache_read(p, h->e4m3, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

attn_status attn_cache_poll_device_error(attn_cache_handle h, int* code) {
    if (!h || !code) return ATTN_ERR_INVALID_ARG;
    *code = 0;
    if (cudaDeviceSynchronize() != cudaSuccess) return ATTN_ERR_CUDA;
    if (cudaMemcpy(code, h->c.err, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return ATTN_ERR_CUDA;
    if (*code != 0 && !clear_error(h->c.err)) return ATTN_ERR_CUDA;
    return *code == 0 ? ATTN_OK : *code & attn::kCacheErrWait ? ATTN_ERR_DEVICE_TIMEOUT : ATTN_ERR_INVALID_ARG;
}

attn_status attn_cache_destroy(attn_cache_handle h) {
    if (!h) return ATTN_OK;
    const cudaError_t e = cudaDeviceSynchronize();
    if (h->c.err) cudaFree(h->c.err);
    delete h;
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

attn_status attn_paged_create(attn_paged_handle* out, int B, int Hq, int Hkv, int S_q, int d, float scale,
                              attn_mask_kind kind, int window) {
    if (!out) return ATTN_ERR_INVALID_ARG;
    *out = nullptr;
    if (!std::isfinite(scale) || !(scale > 0.f)) return ATTN_ERR_INVALID_ARG;
    const attn_status vs = validate_paged(B, Hq, Hkv, S_q, kind, window);
    if (vs != ATTN_OK) return vs;
    if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
    attn_paged_plan* h = new (std::nothrow) attn_paged_plan();
    if (!h) return ATTN_ERR_OOM;
    h->B = B; h->Hq = Hq; h->Hkv = Hkv; h->S_q = S_q; h->d = d; h->kind = kind; h->scale = scale;
    h->window = window_of(kind, window);
    auto fail = [&](cudaError_t e) {
        free_paged(h);
        return e == cudaErrorMemoryAllocation ? ATTN_ERR_OOM : ATTN_ERR_CUDA;
    };
    cudaError_t e = cudaGetDevice(&h->device);
    if (e != cudaSuccess) return fail(e);
    if ((h->n_sm = attn::current_sm_count()) < 1) return fail(cudaErrorUnknown);
    // room for either type of cache
    const size_t grid = (size_t)h->n_sm * attn::kPagedMostCtasPerSm;
    const size_t rows = 2 * grid * attn::paged_rows_pad(Hq / Hkv * S_q, false);
    if ((e = cudaMalloc(reinterpret_cast<void**>(&h->d_part), rows * d * sizeof(float))) != cudaSuccess) return fail(e);
    if ((e = cudaMalloc(reinterpret_cast<void**>(&h->d_ml), rows * sizeof(float2))) != cudaSuccess) return fail(e);
    if ((e = cudaMalloc(reinterpret_cast<void**>(&h->d_cut), sizeof(int2) * grid)) != cudaSuccess) return fail(e);
    *out = h;
    return ATTN_OK;
}

attn_status attn_paged_forward(attn_paged_handle h, attn_cache_handle cache, const void* Q, const int* page_table,
                               long long table_stride, int max_pages, const int* cache_len, void* O, float* LSE,
                               void* stream) {
    if (!h || !cache || !Q || !O || !aligned(Q, 16) || !aligned(O, 16) || !aligned(LSE, 4)) return ATTN_ERR_INVALID_ARG;
    if (!table_ok(page_table, table_stride, max_pages, cache_len)) return ATTN_ERR_INVALID_ARG;
    if (cache->c.Hkv != h->Hkv || cache->c.d != h->d || cache->device != h->device || !on_device(h->device))
        return ATTN_ERR_INVALID_ARG;
    const attn::PagedShape shape = attn::paged_shape(h->d, cache->e4m3);
    const long long room = (long long)max_pages * cache->c.page;
    const int units = h->Hkv * attn::paged_row_blocks(h->Hq / h->Hkv * h->S_q, cache->e4m3);
    const long long most = shape.least + shape.overhead + room / shape.keys + 1;  // a unit's cost
    // positions, and places on the cost line, fit an int
    if (room > attn::kPagedMostPositions || most * h->B * units > 0x7FFFFFFFLL) return ATTN_ERR_UNSUPPORTED;
    attn::PagedParams p{};
    p.tm = cache->map;
    p.q = Q; p.o = O; p.lse = LSE;
    p.c = cache->c;
    p.t.pages = page_table; p.t.len = cache_len; p.t.stride = table_stride; p.t.max_pages = max_pages;
    p.part_o = h->d_part; p.part_ml = h->d_ml; p.cut = h->d_cut;
    p.B = h->B; p.Hq = h->Hq; p.Hkv = h->Hkv; p.S_q = h->S_q; p.rows = h->Hq / h->Hkv * h->S_q;
    p.units = units;
    p.window = h->window;
    p.causal = h->kind != ATTN_MASK_FULL;
    p.scale_log2 = (float)((double)h->scale * 1.4426950408889634);
    p.watchdog_ns = h->watchdog_ns;
    p.withhold = h->withhold;
    p.box_rows = cache->box_rows;
    const int rows_pad = attn::paged_rows_pad(p.rows, cache->e4m3);
    const int grid = std::min(h->n_sm * attn::paged_ctas_per_sm(p.rows, cache->e4m3), h->grid_limit);
    p.by_unit = (long long)h->B * units <= grid;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = cache->e4m3 ? attn::launch_paged_e4m3(p, grid, st) : attn::launch_paged_bf16(p, grid, st);
    if (e == cudaSuccess && attn::paged_may_cut((long long)h->B * units, room, grid, shape))
        e = attn::launch_paged_merge(p, grid, rows_pad, st);
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

attn_status attn_paged_set_grid_limit(attn_paged_handle h, int max_ctas) {
    if (!h || max_ctas < 1) return ATTN_ERR_INVALID_ARG;
    h->grid_limit = max_ctas;
    return ATTN_OK;
}

attn_status attn_paged_set_watchdog(attn_paged_handle h, long long limit_ns, int withhold) {
    if (!h || limit_ns <= 0 || withhold < 0) return ATTN_ERR_INVALID_ARG;
    h->watchdog_ns = limit_ns;
    h->withhold = withhold;
    return ATTN_OK;
}

attn_status attn_paged_destroy(attn_paged_handle h) {
    if (!h) return ATTN_OK;
    const cudaError_t e = cudaDeviceSynchronize();
    free_paged(h);
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

attn_status attn_paged_split_host(int B, int Hkv, int S_q, int d, attn_dtype dtype, attn_mask_kind kind, int window,
                                  const int* cache_len, int grid, int* n_cta, int* parts, int cap,
                                  int* n_parts) {
    if (!cache_len || !n_cta || !n_parts || grid < 1 || (cap > 0 && !parts))
        return ATTN_ERR_INVALID_ARG;
    const attn_status vs = validate_paged(B, Hkv, Hkv, S_q, kind, window);
    if (vs != ATTN_OK) return vs;
    if ((dtype != ATTN_BF16 && dtype != ATTN_FP8_E4M3) || (d != 64 && d != 128)) return ATTN_ERR_INVALID_ARG;
    const int w = window_of(kind, window);
    const attn::PagedShape shape = attn::paged_shape(d, dtype == ATTN_FP8_E4M3);
    std::vector<unsigned> cost;
    std::vector<int> n;
    try {
        cost.assign(B + 1, 0);
        n.assign(B, 0);
    } catch (...) {
        return ATTN_ERR_OOM;
    }
    unsigned units = 0;
    for (int b = 0; b < B; ++b) {
        int lo, hi;
        if (cache_len[b] < 0) return ATTN_ERR_INVALID_ARG;
        if (cache_len[b] > attn::kPagedMostPositions) return ATTN_ERR_UNSUPPORTED;
        attn::paged_blocks(cache_len[b], S_q, w, shape.keys, lo, hi);
        n[b] = hi - lo;
        if (n[b]) units += Hkv;
        if ((long long)attn::paged_cost(n[b], shape) * Hkv + cost[b] > 0x7FFFFFFFLL) return ATTN_ERR_UNSUPPORTED;
        cost[b + 1] = cost[b] + Hkv * attn::paged_cost(n[b], shape);
    }
    const unsigned W = cost[B];
    const attn::PagedCuts cuts(W, units, grid, shape);
    *n_cta = W ? cuts.C : 0;
    *n_parts = 0;
    for (int c = 0; c < *n_cta; ++c) {
        unsigned at = cuts.begin(c);
        const unsigned end = cuts.begin(c + 1);
        int b = 0;
        while (at < end) {
            while (cost[b + 1] <= at) ++b;
            const unsigned per = attn::paged_cost(n[b], shape), g = (at - cost[b]) / per, off = (at - cost[b]) % per;
            const unsigned to = std::min(per, off + (end - at)), over = shape.overhead;
            const int g0 = std::min<int>(n[b], off > over ? off - over : 0);
            const int g1 = std::min<int>(n[b], to > over ? to - over : 0);
            at += to - off;
            if (g0 >= g1) continue;
            if (cap > 0) {
                if (*n_parts >= cap) return ATTN_ERR_INVALID_ARG;
                const unsigned u0 = cost[b] + g * per + over;
                const int part[8] = {c, b, (int)g, g0, g1, n[b], (int)cuts.owner(u0), (int)cuts.owner(u0 + n[b] - 1)};
                std::copy(part, part + 8, parts + 8 * (size_t)*n_parts);
            }
            ++*n_parts;
        }
    }
    return ATTN_OK;
}

}  // extern "C"
