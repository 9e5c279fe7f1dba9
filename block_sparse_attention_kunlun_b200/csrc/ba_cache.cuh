// Shared definitions of the history-cache kernels (ba_cache.cu: writing,
// reading, page means, page selection; ba_cache_fwd.cu: attention).
//
// The cache holds keys and values as MX blocks (the format of ba_mx.cu): 32
// consecutive values along head_dim share a scale 2^e kept as the byte e + 127,
// each value is an E4M3 code. A page holds page_size slots of every key/value
// head, head by head, so that one head's slots of a page are one contiguous
// piece of memory: elements [num_pages, kv_heads, page_size, head_dim], scales
// [num_pages, kv_heads, page_size, head_dim / 32]. Slot p of sequence b is row
// p % page_size of page page_table[b, p / page_size].
#pragma once

#include "ba_common.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

namespace ba {

struct CacheView {
    uint8_t *k, *v, *k_scales, *v_scales;
    const int32_t *page_table; // [batch, max_pages]
    int *status;               // sticky status word or nullptr
    int32_t batch, max_pages, num_pages, page_shift, kv_heads, head_dim;
};

// A slot or page number outside the cache was met (ba_device_status: BA_ERR_INVALID_ARG).
constexpr int kStatusCacheRange = 4;

__device__ __forceinline__ void cache_range_error(const CacheView &c)
{
    if (c.status) atomicOr(c.status, kStatusCacheRange);
}

// Page number of page index `pi` of sequence b, or -1 (and the status bit) where
// the table has none: every access to the pools goes through this check.
__device__ __forceinline__ int32_t cache_page(const CacheView &c, int32_t b, int32_t pi)
{
    if (pi < 0 || pi >= c.max_pages) return -1;
    const int32_t id = __ldg(c.page_table + int64_t(b) * c.max_pages + pi);
    return id >= 0 && id < c.num_pages ? id : -1;
}

// Row of the pools ([num_pages * kv_heads * page_size] rows of head_dim values)
// of slot `at` (within its page) of head h on page `id`.
__device__ __forceinline__ int64_t cache_row(const CacheView &c, int32_t id, int32_t h, int32_t at)
{
    return ((int64_t(id) * c.kv_heads + h) << c.page_shift) + at;
}

// Sequence that owns row `row` of a jagged batch: the b with offs[b] <= row < offs[b + 1].
__device__ __forceinline__ int32_t sequence_of_row(const int32_t *offs, int32_t batch, int32_t row)
{
    int32_t lo = 0, hi = batch; // offs[lo] <= row < offs[hi]
    while (hi - lo > 1) {
        const int32_t mid = (lo + hi) >> 1;
        if (__ldg(offs + mid) <= row) lo = mid;
        else hi = mid;
    }
    return lo;
}

// 2^(code - 127) for an E8M0 code in [0, 254] (code 0 is the subnormal 2^-127).
__device__ __forceinline__ float mx_scale(uint32_t code)
{
    return __uint_as_float(code ? code << 23 : 0x00400000u);
}

// Two E4M3 codes (the low 16 bits) as floats, exactly.
__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t two)
{
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(two), __NV_E4M3);
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

cudaError_t launch_cache_write(const CacheView &c, bool f32, const void *k, const void *v, const int32_t *row_offsets,
                               const int32_t *starts, int32_t total_rows, int num_sms, cudaStream_t stream);
cudaError_t launch_cache_read(const CacheView &c, bool f32, const int32_t *row_offsets, const int32_t *starts,
                              int32_t total_rows, void *k, void *v, int num_sms, cudaStream_t stream);
cudaError_t launch_cache_summarize(const CacheView &c, const int32_t *starts, const int32_t *ends, float *summaries,
                                   int num_sms, cudaStream_t stream);

// What the page selection and the attention know of the queries.
struct CacheQuery {
    const __nv_bfloat16 *q;      // [rows, kv_heads * group, head_dim]
    const int32_t *q_offsets;    // [batch + 1]
    const int32_t *lens;         // [batch] cached slots
    const int32_t *positions;    // [rows] or nullptr: lens + index within the sequence
    int32_t rows, group, block, window;
};

// Position of row t (of n, first row at global row q0) of a sequence with len cached slots.
__device__ __forceinline__ int32_t query_position(const CacheQuery &q, int32_t q0, int32_t len, int32_t t)
{
    return q.positions ? __ldg(q.positions + q0 + t) : len + t;
}

// First position the block rule shows to a query at `pos`, in 32 bits (pos >= 0).
__device__ __forceinline__ int32_t rule_start(const CacheQuery &q, int32_t pos)
{
    return int32_t(window_start(pos, q.block, q.window));
}

// The most pages of a sequence that the selection can rank: one row's keys (8 bytes a
// page) stay in shared memory.
constexpr int32_t kSelectMaxPages = 16384;

cudaError_t launch_cache_select(const CacheView &c, const CacheQuery &q, const float *summaries, int32_t topk,
                                uint32_t *page_mask, cudaStream_t stream);

struct CacheFwd {
    CacheView c;
    CacheQuery q;
    const uint32_t *tree;      // [rows, tree_words] or nullptr (chain)
    const uint32_t *page_mask; // [rows, kv_heads, ceil(max_pages / 32)] or nullptr
    int32_t tree_words, mask_words;
    int32_t chunk, nsplit;     // cached slots a split covers (the last one takes the rest)
    float scale_log2;          // log2(e) / sqrt(head_dim)
    __nv_bfloat16 *out;
    float *lse;                // [heads, rows]
    float2 *part_ml;           // [nsplit, rows * heads] running maximum (log2) and sum
    float *part_o;             // [nsplit, rows * heads, head_dim]
};

// How the attention is cut up; a function of host values alone, so that the workspace
// query and the call agree.
struct CacheFwdPlan {
    int32_t tile_rows; // query rows (token, head of the group) a block takes at once
    int32_t chunk, nsplit;
    int64_t tiles;
    size_t bytes;
};
CacheFwdPlan cache_fwd_plan(int32_t batch, int32_t rows, int32_t kv_heads, int32_t group, int32_t head_dim,
                            int64_t slots, int32_t page_size, int64_t block, int64_t window,
                            bool has_mask);
cudaError_t launch_cache_fwd(const CacheFwd &p, const CacheFwdPlan &plan, cudaStream_t stream);

} // namespace ba
