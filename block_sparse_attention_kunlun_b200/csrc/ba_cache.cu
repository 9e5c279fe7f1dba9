// The history cache's memory-bound kernels (layout and format in ba_cache.cuh):
//   cache_write_kernel      dense rows, quantised as they are written
//   cache_read_kernel       slots back as dense rows
//   cache_summarize_kernel  the mean key of each full page
//   cache_select_kernel     the pages whose mean keys score highest for a query
// "GEM (Meta)", section "Training infrastructure", has the jagged histories;
// the pages do not describe how they are served.
#include "ba_cache.cuh"
#include "ba_kernels.cuh"
#include "ba_ptx.cuh"

#include <type_traits>

namespace ba {

namespace {

constexpr int kRowThreads = 256;
constexpr int kRowsPerBlock = 32; // most dense rows a block takes

// Pool rows (head 0) of `n` consecutive dense rows from row0 on. A row whose slot is
// not in the cache gets -1.
__device__ __forceinline__ void find_rows(const CacheView &c, const int32_t *row_offsets, const int32_t *starts,
                                          int32_t row0, int32_t n, int64_t *target)
{
    if (int(threadIdx.x) < n) {
        const int32_t row = row0 + threadIdx.x;
        const int32_t b = sequence_of_row(row_offsets, c.batch, row);
        const int64_t slot = int64_t(__ldg(starts + b)) + row - __ldg(row_offsets + b);
        const int64_t pi = slot >> c.page_shift;
        const int32_t id = slot >= 0 && pi < c.max_pages ? cache_page(c, b, int32_t(pi)) : -1;
        if (id < 0) cache_range_error(c);
        target[threadIdx.x] = id < 0 ? -1 : cache_row(c, id, 0, int32_t(slot & ((1 << c.page_shift) - 1)));
    }
    __syncthreads();
}

// Eight values from a dense row.
__device__ __forceinline__ void load8(const __nv_bfloat16 *x, float (&f)[8])
{
    const uint4 w = __ldcs(reinterpret_cast<const uint4 *>(x));
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(ws[i] << 16);
        f[2 * i + 1] = __uint_as_float(ws[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void load8(const float *x, float (&f)[8])
{
    const float4 a = __ldcs(reinterpret_cast<const float4 *>(x)), b = __ldcs(reinterpret_cast<const float4 *>(x) + 1);
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}

} // namespace

// x / d for the head number: by a multiplication with ceil(2^32 / d), exact while x d < 2^32
// (x < 32 d here), or magic = 0 and a division.
__device__ __forceinline__ uint32_t div_heads(uint32_t x, uint32_t d, uint32_t magic)
{
    return magic ? __umulhi(x, magic) : x / d;
}

// D / 8 lanes hold a (row, head), eight values each, four lanes one 32-value block: 16 (or 32)
// bytes in, 8 bytes out per lane, so a warp reads 512 (1024) and writes 256 consecutive bytes
// of rows and pages. The block's largest magnitude takes two shuffles; e = floor(log2 amax) - 8
// is its exponent field, and multiplying by 2^-e is exact in float32 (the quotient stays below
// 2^9; what underflows is far below E4M3's smallest value), so the conversion to E4M3 is the
// only rounding. fmaxf drops NaN: a NaN leaves its block's scale alone and becomes E4M3's NaN;
// an infinity gives e = 120 and the largest code.
// Bound by HBM for many rows (each thread has kBatch loads under way): whole jagged histories
// of 540,000 rows of 8 heads of 128 in bf16, 3.3 GB, in 553 to 585 us, 5.7 to 6.0 TB/s. For few rows
// by latency: one event for each of 256 histories takes 4.7 us within a captured step (9.2 with its call).
template <typename T, int D>
__global__ void __launch_bounds__(kRowThreads)
    cache_write_kernel(const CacheView c, const T *__restrict__ k, const T *__restrict__ v,
                       const int32_t *__restrict__ row_offsets, const int32_t *__restrict__ starts, int32_t total_rows,
                       int32_t rows_per_block, uint32_t magic)
{
    constexpr int L = D / 8, kStep = kRowThreads / L, kBatch = 4;
    __shared__ int64_t target[kRowsPerBlock];
    const int32_t row0 = blockIdx.x * rows_per_block;
    // (rows behind the last sequence are nobody's)
    const int32_t n = min(rows_per_block, min(total_rows, __ldg(row_offsets + c.batch)) - row0);
    if (n <= 0) return;
    find_rows(c, row_offsets, starts, row0, n, target);
    const bool values = blockIdx.y != 0;
    const int d8 = threadIdx.x % L;
    const T *src = (values ? v : k) + int64_t(row0) * c.kv_heads * D + d8 * 8;
    uint8_t *elems = values ? c.v : c.k, *scales = values ? c.v_scales : c.k_scales;
    const uint32_t heads = c.kv_heads, all = n * heads;
    for (uint32_t x0 = 0; x0 < all; x0 += kBatch * kStep) {
        float f[kBatch][8];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const uint32_t x = x0 + i * kStep + threadIdx.x / L;
            if (x < all) {
                load8(src + int64_t(x) * D, f[i]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) f[i][j] = 0.f;
            }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const uint32_t x = x0 + i * kStep + threadIdx.x / L;
            float amax = fmaxf(fmaxf(fmaxf(fabsf(f[i][0]), fabsf(f[i][1])), fmaxf(fabsf(f[i][2]), fabsf(f[i][3]))),
                               fmaxf(fmaxf(fabsf(f[i][4]), fabsf(f[i][5])), fmaxf(fabsf(f[i][6]), fabsf(f[i][7]))));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            // exponent code e + 127 = field - 8, not below 0 (subnormal maxima too); an all-zero block has e = -8
            uint32_t code = __float_as_uint(amax) >> 23;
            code = amax > 0.f ? (code > 8 ? code - 8 : 0u) : 119u;
            const float inv = __uint_as_float(code < 254 ? (254 - code) << 23 : 0x00400000u);
            uint32_t w[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float *g = f[i] + 4 * j;
                const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(g[0] * inv, g[1] * inv), __NV_SATFINITE, __NV_E4M3);
                const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(g[2] * inv, g[3] * inv), __NV_SATFINITE, __NV_E4M3);
                w[j] = lo | (hi << 16);
            }
            // the head's scale codes as one word (two or four bytes), gathered by its first lane
            uint32_t word = code << (8 * (d8 / 4));
            word |= __shfl_xor_sync(0xffffffffu, word, 4);
            if (D == 128) word |= __shfl_xor_sync(0xffffffffu, word, 8);
            if (x >= all) continue;
            const uint32_t r = div_heads(x, heads, magic), h = x - r * heads;
            if (target[r] < 0) continue;
            const int64_t row = target[r] + (int64_t(h) << c.page_shift);
            *reinterpret_cast<uint2 *>(elems + row * D + d8 * 8) = make_uint2(w[0], w[1]);
            if (d8 == 0) {
                if (D == 128) *reinterpret_cast<uint32_t *>(scales + row * 4) = word;
                else *reinterpret_cast<uint16_t *>(scales + row * 2) = uint16_t(word);
            }
        }
    }
}

// D / 16 lanes hold a (row, head), sixteen values each: 16 bytes of codes in, 32 (bf16) or 64
// bytes out. A bf16 result is exact (four significant bits) unless it falls below bf16's
// normal range. Bound by HBM: 65,000 rows of 8 heads of 128 as bf16, 0.41 GB, in 71 us, 5.7
// TB/s; as float32 (0.085 GB) 18 us (14 within a captured step), with 16-byte stores 25.
template <typename T, int D>
__global__ void __launch_bounds__(kRowThreads)
    cache_read_kernel(const CacheView c, const int32_t *__restrict__ row_offsets, const int32_t *__restrict__ starts,
                      int32_t total_rows, int32_t rows_per_block, uint32_t magic, T *__restrict__ k, T *__restrict__ v)
{
    constexpr int L = D / 16, kStep = kRowThreads / L, kBatch = 2;
    __shared__ int64_t target[kRowsPerBlock];
    const int32_t row0 = blockIdx.x * rows_per_block;
    // (rows behind the last sequence are nobody's)
    const int32_t n = min(rows_per_block, min(total_rows, __ldg(row_offsets + c.batch)) - row0);
    if (n <= 0) return;
    find_rows(c, row_offsets, starts, row0, n, target);
    const bool values = blockIdx.y != 0;
    const int d16 = threadIdx.x % L;
    T *dst = (values ? v : k) + int64_t(row0) * c.kv_heads * D + d16 * 16;
    const bool wide = reinterpret_cast<uintptr_t>(dst) % 32 == 0; // (16-byte aligned tensors may be neither)
    const uint8_t *elems = values ? c.v : c.k, *scales = values ? c.v_scales : c.k_scales;
    const uint32_t heads = c.kv_heads, all = n * heads;
    for (uint32_t x0 = threadIdx.x / L; x0 < all; x0 += kBatch * kStep) {
        uint4 w[kBatch];
        uint32_t code[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const uint32_t x = x0 + i * kStep;
            w[i] = make_uint4(0u, 0u, 0u, 0u);
            code[i] = 127;
            if (x < all) {
                const uint32_t r = div_heads(x, heads, magic), h = x - r * heads;
                if (target[r] >= 0) {
                    const int64_t row = target[r] + (int64_t(h) << c.page_shift);
                    w[i] = __ldg(reinterpret_cast<const uint4 *>(elems + row * D) + d16);
                    code[i] = __ldg(scales + row * (D / 32) + d16 / 2);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const uint32_t x = x0 + i * kStep;
            if (x >= all) break;
            const float s = mx_scale(code[i]);
            const uint32_t ws[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
            uint32_t o[4 * sizeof(T)];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float2 f = e4m3x2_to_f32((ws[j / 2] >> (16 * (j % 2))) & 0xffffu);
                f.x *= s;
                f.y *= s;
                if constexpr (sizeof(T) == 2) {
                    o[j] = pack_bf16x2(f.x, f.y);
                } else {
                    o[2 * j] = __float_as_uint(f.x);
                    o[2 * j + 1] = __float_as_uint(f.y);
                }
            }
            T *const out = dst + int64_t(x) * D;
            if (wide) { // whole sectors a store
#pragma unroll
                for (int j = 0; j < int(sizeof(T)) / 2; ++j) st_global_32b(out + j * (32 / sizeof(T)), o + 8 * j);
            } else {
#pragma unroll
                for (int j = 0; j < int(sizeof(T)); ++j)
                    __stcs(reinterpret_cast<uint4 *>(out) + j,
                           make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]));
            }
        }
    }
}

namespace {

// Rows a block takes: enough blocks to fill the GPU when there are few rows (a step of
// single events), up to 32 rows a block when there are many.
int32_t rows_per_block(int32_t total_rows, int num_sms)
{
    const int64_t want = (int64_t(total_rows) + 2 * num_sms - 1) / (2 * num_sms);
    return int32_t(want < 1 ? 1 : (want > kRowsPerBlock ? kRowsPerBlock : want));
}

} // namespace

namespace {

uint32_t heads_magic(int32_t heads)
{
    return heads > 1 && heads <= 8192 ? uint32_t(((uint64_t(1) << 32) + heads - 1) / heads) : 0;
}

template <typename T, int D>
void launch_write(const CacheView &c, const void *k, const void *v, const int32_t *row_offsets, const int32_t *starts,
                  int32_t total_rows, int32_t rpb, cudaStream_t stream)
{
    cache_write_kernel<T, D><<<dim3((total_rows + rpb - 1) / rpb, 2), kRowThreads, 0, stream>>>(
        c, static_cast<const T *>(k), static_cast<const T *>(v), row_offsets, starts, total_rows, rpb,
        heads_magic(c.kv_heads));
}

template <typename T, int D>
void launch_read(const CacheView &c, const int32_t *row_offsets, const int32_t *starts, int32_t total_rows, void *k,
                 void *v, int32_t rpb, cudaStream_t stream)
{
    cache_read_kernel<T, D><<<dim3((total_rows + rpb - 1) / rpb, 2), kRowThreads, 0, stream>>>(
        c, row_offsets, starts, total_rows, rpb, heads_magic(c.kv_heads), static_cast<T *>(k), static_cast<T *>(v));
}

} // namespace

cudaError_t launch_cache_write(const CacheView &c, bool f32, const void *k, const void *v, const int32_t *row_offsets,
                               const int32_t *starts, int32_t total_rows, int num_sms, cudaStream_t stream)
{
    const int32_t rpb = rows_per_block(total_rows, num_sms);
    if (f32 && c.head_dim == 64) launch_write<float, 64>(c, k, v, row_offsets, starts, total_rows, rpb, stream);
    else if (f32) launch_write<float, 128>(c, k, v, row_offsets, starts, total_rows, rpb, stream);
    else if (c.head_dim == 64)
        launch_write<__nv_bfloat16, 64>(c, k, v, row_offsets, starts, total_rows, rpb, stream);
    else launch_write<__nv_bfloat16, 128>(c, k, v, row_offsets, starts, total_rows, rpb, stream);
    return cudaGetLastError();
}

cudaError_t launch_cache_read(const CacheView &c, bool f32, const int32_t *row_offsets, const int32_t *starts,
                              int32_t total_rows, void *k, void *v, int num_sms, cudaStream_t stream)
{
    const int32_t rpb = rows_per_block(total_rows, num_sms);
    if (f32 && c.head_dim == 64) launch_read<float, 64>(c, row_offsets, starts, total_rows, k, v, rpb, stream);
    else if (f32) launch_read<float, 128>(c, row_offsets, starts, total_rows, k, v, rpb, stream);
    else if (c.head_dim == 64) launch_read<__nv_bfloat16, 64>(c, row_offsets, starts, total_rows, k, v, rpb, stream);
    else launch_read<__nv_bfloat16, 128>(c, row_offsets, starts, total_rows, k, v, rpb, stream);
    return cudaGetLastError();
}

// One warp per (page, head): its slots are page_size * head_dim consecutive bytes, read 16
// bytes a lane, eight loads at a time; each lane sums its sixteen columns over its rows in
// float32 and the lanes that share columns are added at the end. The pages of a (sequence,
// head) are dealt to `share` warps, as many as the GPU holds at 128 registers a thread. Bound by
// one page's latency for few pages (8.2 us for one of each of 256 histories, 7.2 within a captured
// step); for many by HBM: 0.29 GB of keys in 50 to 55 us, 5.3 to 5.8 TB/s (60 with each batch loaded
// after the one before it was summed; 112 squeezed into 96 registers for more warps).
template <int D>
__global__ void __launch_bounds__(128)
    cache_summarize_kernel(const CacheView c, const int32_t *__restrict__ starts, const int32_t *__restrict__ ends,
                           int32_t share, float *__restrict__ summaries)
{
    constexpr int kLanes = D / 16, kRows = 32 / kLanes, kBatch = 8; // lanes of a row, rows of a load
    const int lane = threadIdx.x & 31;
    const int64_t unit = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 5);
    const int32_t pair = int32_t(unit / share), part = int32_t(unit % share);
    const int32_t b = pair / c.kv_heads, h = pair % c.kv_heads;
    if (b >= c.batch) return;
    const int32_t first = max(__ldg(starts + b), 0) >> c.page_shift;
    const int32_t end = max(__ldg(ends + b), 0) >> c.page_shift; // pages below are full
    if (end > c.max_pages && part == 0 && h == 0 && lane == 0) cache_range_error(c);
    const int32_t stop = min(end, c.max_pages);
    const int32_t loads = (1 << c.page_shift) / kRows; // of a page: 2 .. 32
    const int col = lane % kLanes;
    const float inv = 1.f / float(1 << c.page_shift); // a power of two
    // this warp's pages: the number of the next one, and the next batch's loads, are under way
    // while a batch is summed
    auto page_at = [&](int32_t &pi) { // the next page that has a number, from pi on
        for (; pi < stop; pi += share) {
            const int32_t id = cache_page(c, b, pi);
            if (id >= 0) return id;
            if (lane == 0) cache_range_error(c);
        }
        return -1;
    };
    uint4 w[kBatch], w2[kBatch];
    uint32_t code[kBatch], code2[kBatch];
    auto load = [&](int32_t id, int32_t u0, uint4 (&x)[kBatch], uint32_t (&y)[kBatch]) {
        const int64_t row0 = cache_row(c, id, h, 0);
        const uint4 *src = reinterpret_cast<const uint4 *>(c.k + row0 * D) + lane;
        const uint8_t *sc = c.k_scales + (row0 + lane / kLanes) * (D / 32) + col / 2;
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            if (u0 + u < loads) {
                x[u] = __ldg(src + (u0 + u) * 32);
                y[u] = __ldg(sc + (u0 + u) * kRows * (D / 32));
            }
    };
    int32_t pi = first + part, id = page_at(pi);
    if (id >= 0) load(id, 0, w, code);
    while (id >= 0) {
        pi += share;
        const int32_t next = page_at(pi);
        float2 acc[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = make_float2(0.f, 0.f);
        for (int32_t u0 = 0; u0 < loads; u0 += kBatch) {
            if (u0 + kBatch < loads) load(id, u0 + kBatch, w2, code2);
            else if (next >= 0) load(next, 0, w2, code2);
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
                if (u0 + u < loads) {
                    const uint32_t ws[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
                    const float s = mx_scale(code[u]);
                    const float2 s2 = make_float2(s, s);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        acc[i] = ffma2(e4m3x2_to_f32((ws[i / 2] >> (16 * (i % 2))) & 0xffffu), s2, acc[i]);
                }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                w[u] = w2[u];
                code[u] = code2[u];
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
#pragma unroll
            for (int m = kLanes; m < 32; m <<= 1) {
                acc[i].x += __shfl_xor_sync(0xffffffffu, acc[i].x, m);
                acc[i].y += __shfl_xor_sync(0xffffffffu, acc[i].y, m);
            }
        }
        if (lane < kLanes) {
            float4 *dst = reinterpret_cast<float4 *>(summaries + (int64_t(id) * c.kv_heads + h) * D) + col * 4;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                dst[i] = make_float4(acc[2 * i].x * inv, acc[2 * i].y * inv, acc[2 * i + 1].x * inv,
                                     acc[2 * i + 1].y * inv);
        }
        id = next;
    }
}

cudaError_t launch_cache_summarize(const CacheView &c, const int32_t *starts, const int32_t *ends, float *summaries,
                                   int num_sms, cudaStream_t stream)
{
    // as many warps as the GPU holds, whatever the number of (sequence, head) pairs
    const int64_t pairs = int64_t(c.batch) * c.kv_heads;
    int64_t share = (int64_t(num_sms) * 16 + pairs - 1) / pairs;
    if (share > c.max_pages) share = c.max_pages;
    const int64_t blocks = (pairs * share + 3) / 4;
    if (c.head_dim == 64)
        cache_summarize_kernel<64><<<unsigned(blocks), 128, 0, stream>>>(c, starts, ends, int32_t(share), summaries);
    else
        cache_summarize_kernel<128><<<unsigned(blocks), 128, 0, stream>>>(c, starts, ends, int32_t(share), summaries);
    return cudaGetLastError();
}

namespace {

// Scores as numbers that order like them; NaN below every number, and 0 is left for pages that
// are no candidates. -0 becomes +0.
__device__ __forceinline__ uint64_t score_key(double s)
{
    if (s != s) return 1;
    const uint64_t b = uint64_t(__double_as_longlong(s + 0.0));
    return (b >> 63) ? ~b : b | (uint64_t(1) << 63);
}
__device__ __forceinline__ uint32_t score_key(float s)
{
    if (s != s) return 1;
    const uint32_t b = __float_as_uint(s + 0.f);
    return (b >> 31) ? ~b : b | (1u << 31);
}
__device__ __forceinline__ float key_score(uint32_t key)
{
    return __uint_as_float(key >> 31 ? key & 0x7fffffffu : ~key);
}

__device__ __forceinline__ uint32_t warp_max(uint32_t x) { return __reduce_max_sync(0xffffffffu, x); }
__device__ __forceinline__ uint32_t warp_min(uint32_t x) { return __reduce_min_sync(0xffffffffu, x); }
__device__ __forceinline__ uint64_t warp_max(uint64_t x)
{
#pragma unroll
    for (int m = 16; m; m >>= 1) x = max(x, __shfl_xor_sync(0xffffffffu, x, m));
    return x;
}
__device__ __forceinline__ uint64_t warp_min(uint64_t x)
{
#pragma unroll
    for (int m = 16; m; m >>= 1) x = min(x, __shfl_xor_sync(0xffffffffu, x, m));
    return x;
}

// The keys key[0 .. most) of one row as a warp meets them: held in registers (kHeld a lane) or
// read again each time (kHeld = 0).
template <typename K, int kHeld>
struct Keys {
    const K *key;
    int32_t most;
    K held[kHeld > 0 ? kHeld : 1];

    __device__ __forceinline__ Keys(const K *k, int32_t n) : key(k), most(n)
    {
        const int lane = threadIdx.x & 31;
        if constexpr (kHeld > 0) {
#pragma unroll
            for (int i = 0; i < kHeld; ++i) held[i] = i * 32 + lane < n ? k[i * 32 + lane] : 0;
        }
    }
    template <typename F>
    __device__ __forceinline__ void each(F f) const
    {
        if constexpr (kHeld > 0) {
#pragma unroll
            for (int i = 0; i < kHeld; ++i) f(held[i]);
        } else {
            for (int32_t p = threadIdx.x & 31; p < most; p += 32) f(key[p]);
        }
    }
    // keys at or above x (x > 0), over the warp
    __device__ __forceinline__ int32_t count(K x) const
    {
        int32_t n = 0;
        each([&](K y) { n += y >= x; });
        return __reduce_add_sync(0xffffffffu, n);
    }
    // The largest x with at least topk keys at or above it, or any x with exactly topk of them
    // (count then says topk). The caller has made sure that there are more than topk candidates.
    // Found bit by bit from the keys' highest differing bit down.
    __device__ __forceinline__ K edge(int32_t topk, int32_t &count_at) const
    {
        constexpr int kTop = sizeof(K) * 8 - 1;
        K top = 0, low = ~K(0);
        each([&](K x) {
            top = max(top, x);
            low = min(low, x ? x : ~K(0));
        });
        top = warp_max(top);
        low = warp_min(low);
        const K diff = top ^ low;
        int bit = sizeof(K) == 8 ? 63 - __clzll((long long)diff) : 31 - __clz(int(diff)); // -1: all alike
        K x = bit < 0 ? top : bit == kTop ? 0 : top >> (bit + 1) << (bit + 1);             // the common prefix
        count_at = -1;
        for (; bit >= 0 && count_at != topk; --bit) {
            const K trial = x | K(1) << bit;
            const int32_t n = count(trial);
            if (n >= topk) {
                x = trial;
                count_at = n;
            }
        }
        return x;
    }
};

// Bits of the keys above `edge`, and of the first `equal` of those equal to it.
template <typename K>
__device__ __forceinline__ void write_bits(const K *key, int32_t most, K edge, int32_t equal, uint32_t *dst,
                                           int32_t words)
{
    const int lane = threadIdx.x & 31;
    int32_t seen = 0;
    for (int32_t w = 0; w < words; ++w) {
        const int32_t p = w * 32 + lane;
        const K x = p < most ? key[p] : 0;
        const bool even = x == edge && x != 0;
        const uint32_t ties = __ballot_sync(0xffffffffu, even);
        const int32_t rank = seen + __popc(ties & ((1u << lane) - 1));
        const uint32_t word = __ballot_sync(0xffffffffu, x > edge || (even && rank < equal));
        seen += __popc(ties);
        if (lane == 0) dst[w] = word;
    }
}

// a warp a row for the final choice, and four for one row
__host__ __device__ constexpr int select_warps(int rows) { return rows > 4 ? rows : 4; }

__device__ __forceinline__ void select_mma(float (&c)[4], const uint32_t (&a)[4], uint2 b)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b.x), "r"(b.y));
}

// Two values as bf16 and what is left of them, as bf16 too: a = hi + lo up to 2^-16 |a|.
__device__ __forceinline__ void split_bf16x2(float a, float b, uint32_t &hi, uint32_t &lo)
{
    hi = pack_bf16x2(a, b);
    lo = pack_bf16x2(a - __uint_as_float(hi << 16), b - __uint_as_float(hi & 0xffff0000u));
}

} // namespace

// Scores of the candidate pages for kRows rows of one (sequence, key/value head), then the
// topk of each. Which of two pages wins is decided by the scores in float64 (the products of
// bf16 queries and float32 means are exact there, the sums off by some 2^-53, so the choice
// does not hang on the order of summation), but few pages need one: all scores are formed
// less exactly, off by at most E, so with tau the topk-th largest of them, pages above tau + 2 E
// are in, pages below tau - 2 E out, and only when more than topk pages reach tau - 2 E are
// those in between scored again in float64. (All in float64: 50 us for the scores alone in the
// case below; DFMA chains, not bandwidth, were the bound.)
//
// The scores are warp-wide MMAs of 16 pages by 8 rows. Means and sums of queries are split in
// two bf16 each, m = m1 + m2 and q = q1 + q2 up to 2^-16 of their size, and m1 q1 + m2 q1 + m1 q2
// are added up in float32 (q2 is 0 for a group of one head, whose queries are bf16 already).
// With A = sum |q| and M = max |mean|, each MMA's 16 products and its sum so far, all below A M,
// lose at most 18 2^-23 A M (cut, not rounded), the splits 2^-16 A M for each product of rests
// that is left out, the rounding of q to float32 2^-24 A M: E is their sum, 1.01 for E's own
// roundings, and an absolute part for what underflows. A lane's four consecutive columns of
// its two pages are its columns of an MMA step, so the means go from memory to the MMAs
// through registers alone. (Float32 on the CUDA cores, one page a lane, means through shared
// memory and a tighter band: 45 us where this takes 27, for 8 trees of 17 to 64 rows over
// 16,000 to 33,000 events in 64-slot pages, 8 heads of 128, the 32 best pages.) No unit is busy
// half of the time there. Offsets, page numbers, means and the choice follow one another in each
// block, some 8 us of the 27; and every block of eight rows reads all candidates' means of its
// sequence and head again, some 70 MB through L2 where 12.5 MB differ. Three blocks of eight rows
// an SM (up to some 1100 pages, whose keys take 70 KB a block), at the price of a few spilled registers:
// with two 32 us. Rows go to blocks of four warps one by one (eight: 15.5 for 14.0 us, 64 histories).
template <int D, int kRows>
__global__ void __launch_bounds__(select_warps(kRows) * 32, kRows > 1 ? 3 : 4)
    cache_select_kernel(const CacheView c, const CacheQuery q, const float *__restrict__ summaries, int32_t topk,
                        uint32_t *__restrict__ page_mask)
{
    constexpr int kSteps = D / 16, kWarps = select_warps(kRows);
    extern __shared__ __align__(16) uint64_t keys[]; // [kRows][max_pages]: float32 keys in a row's first half
    __shared__ uint2 q_hi[kSteps][32], q_lo[kSteps][32]; // the rows' sums over the group, as MMA fragments
    __shared__ float q_abs[kSteps][8];               // sums of their magnitudes
    __shared__ int32_t cands[kRows];
    __shared__ uint32_t max_mean;                    // largest |mean| (its bits)
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t4 = lane & 3;
    const int32_t h = blockIdx.y;
    // the sequence and its tile of kRows rows: tiles are numbered floor(offs[b] / kRows) + b
    // (tiles of one row by their row)
    int32_t b, tile;
    {
        int32_t lo = 0, n = c.batch;
        while (n > 1) {
            const int32_t step = (n + 31) / 32, at = lo + lane * step;
            const bool ok = lane * step < n &&
                            __ldg(q.q_offsets + at) / kRows + (kRows > 1 ? at : 0) <= int32_t(blockIdx.x);
            const int32_t cnt = __popc(__ballot_sync(0xffffffffu, ok));
            n = min(step, n - (cnt - 1) * step);
            lo += (cnt - 1) * step;
        }
        b = lo;
        tile = int32_t(blockIdx.x) - (__ldg(q.q_offsets + b) / kRows + (kRows > 1 ? b : 0));
    }
    const int32_t q0 = __ldg(q.q_offsets + b), n = __ldg(q.q_offsets + b + 1) - q0;
    const int32_t t0 = tile * kRows;
    if (t0 >= n) return;
    const int32_t given = max(__ldg(q.lens + b), 0), len = min(given, c.max_pages << c.page_shift);
    if (given > len && threadIdx.x == 0) cache_range_error(c);
    const int32_t full = len >> c.page_shift; // pages below are full
    if (threadIdx.x < kRows) {
        // candidates of the row: pages that start before its window and are full
        int32_t cand = 0;
        if (t0 + int(threadIdx.x) < n) {
            const int32_t pos = query_position(q, q0, len, t0 + threadIdx.x);
            const int32_t ws = pos >= 0 ? rule_start(q, pos) : 0;
            cand = min(int32_t((int64_t(ws) + (1 << c.page_shift) - 1) >> c.page_shift), full);
        }
        cands[threadIdx.x] = cand;
    }
    if (threadIdx.x == 0) max_mean = 0;
    const __nv_bfloat16 *const q_first = q.q + ((int64_t(q0) + t0) * c.kv_heads + h) * q.group * D;
    const int64_t q_row = int64_t(c.kv_heads) * q.group * D;
    // columns d .. d + 3 of row r's sum over the group
    auto q_sum = [&](int r, int d, double (&s)[4]) {
        s[0] = s[1] = s[2] = s[3] = 0.0;
        const uint2 *src = reinterpret_cast<const uint2 *>(q_first + r * q_row + d);
#pragma unroll 4
        for (int32_t x = 0; x < q.group; ++x) {
            const uint2 w = __ldg(src + x * (D / 4));
            s[0] += double(__uint_as_float(w.x << 16));
            s[1] += double(__uint_as_float(w.x & 0xffff0000u));
            s[2] += double(__uint_as_float(w.y << 16));
            s[3] += double(__uint_as_float(w.y & 0xffff0000u));
        }
    };
    for (int x = warp; x < kSteps; x += kWarps) { // (lane: row g, columns 16 x + 4 t4 ..)
        float f[4] = {0.f, 0.f, 0.f, 0.f};
        if (g < kRows && t0 + g < n) {
            double s[4];
            q_sum(g, 16 * x + 4 * t4, s);
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = float(s[i]);
        }
        uint2 hi, lo;
        split_bf16x2(f[0], f[1], hi.x, lo.x);
        split_bf16x2(f[2], f[3], hi.y, lo.y);
        q_hi[x][lane] = hi;
        q_lo[x][lane] = lo;
        float a = fabsf(f[0]) + fabsf(f[1]) + (fabsf(f[2]) + fabsf(f[3]));
        a += __shfl_xor_sync(0xffffffffu, a, 1);
        a += __shfl_xor_sync(0xffffffffu, a, 2);
        if (t4 == 0) q_abs[x][g] = a;
    }
    __syncthreads();
    int32_t most = 0;
#pragma unroll
    for (int r = 0; r < kRows; ++r) most = max(most, cands[r]);

    const bool grouped = q.group > 1;
    float largest = 0.f;
    const float *const head = summaries + h * D + t4 * 4;
    for (int32_t p0 = warp * 16; p0 < most; p0 += kWarps * 16) {
        int32_t id = -1;
        if (lane < 16 && p0 + lane < most) {
            id = cache_page(c, b, p0 + lane);
            if (id < 0) cache_range_error(c);
        }
        float4 w[2][kSteps]; // of pages p0 + g, p0 + g + 8
        int32_t from[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            from[i] = __shfl_sync(0xffffffffu, id, g + 8 * i);
            const float4 *src = reinterpret_cast<const float4 *>(head + int64_t(from[i]) * (c.kv_heads * D));
#pragma unroll
            for (int x = 0; x < kSteps; ++x)
                w[i][x] = from[i] >= 0 ? __ldg(src + 4 * x) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int x = 0; x < kSteps; ++x) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                largest = fmax3(largest, fabsf(w[i][x].x), fabsf(w[i][x].y));
                largest = fmax3(largest, fabsf(w[i][x].z), fabsf(w[i][x].w));
                split_bf16x2(w[i][x].x, w[i][x].y, hi[i], lo[i]);
                split_bf16x2(w[i][x].z, w[i][x].w, hi[2 + i], lo[2 + i]);
            }
            const uint2 b_hi = q_hi[x][lane];
            select_mma(acc, hi, b_hi);
            select_mma(acc, lo, b_hi);
            if (grouped) select_mma(acc, hi, q_lo[x][lane]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int r = 2 * t4 + (e & 1), p = p0 + g + 8 * (e >> 1);
            if (r < kRows && p < most)
                reinterpret_cast<uint32_t *>(keys + int64_t(r) * c.max_pages)[p] =
                    p < cands[r] && from[e >> 1] >= 0 ? score_key(acc[e]) : 0;
        }
    }
    const uint32_t most_mean = warp_max(__float_as_uint(largest));
    if (lane == 0) atomicMax(&max_mean, most_mean);
    __syncthreads();

    const int32_t words = (c.max_pages + 31) / 32;
    auto choose = [&](int32_t r, auto held) {
        constexpr int kHeld = decltype(held)::value;
        uint64_t *const key64 = keys + int64_t(r) * c.max_pages;
        uint32_t *const key32 = reinterpret_cast<uint32_t *>(key64);
        uint32_t *const dst = page_mask + ((int64_t(q0) + t0 + r) * c.kv_heads + h) * words;
        float bound = 0.f; // sum |q|, then E
#pragma unroll
        for (int x = 0; x < kSteps; ++x) bound += q_abs[x][r];
        const float least = (bound + D * __uint_as_float(max_mean) + D) * 0x1p-120f;
        bound = fmaf(bound * __uint_as_float(max_mean),
                     1.01f * (grouped ? 3 * kSteps * 18 * 0x1p-23f + 3 * 0x1p-16f + 0x1p-24f
                                      : 2 * kSteps * 18 * 0x1p-23f + 0x1p-16f),
                     least);
        uint32_t cut = 1; // pages at or above it are taken, if they are at most topk
        {
            const Keys<uint32_t, kHeld> k(key32, most);
            if (k.count(1) > topk) {
                int32_t at;
                const float tau = key_score(k.edge(topk, at));
                // (not finite: a product or sum overflowed; every candidate is scored again)
                const float low = tau - 2.02f * bound;
                bool fine = fabsf(low) < INFINITY && k.count(score_key(-INFINITY)) == k.count(1);
                cut = fine ? score_key(low) : 1u;
                if (k.count(cut) > topk) {
                    // some stay in doubt: those above the band are in, below it out, in it ranked by
                    // their float64 scores
                    const uint32_t above = fine ? score_key(tau + 2.02f * bound) : ~0u - 1;
                    const int32_t sure = k.count(above + 1), doubts = k.count(cut) - sure;
                    // of four pages at once: eight lanes one
                    auto score = [&](int32_t page) {
                        double s = 0.0;
                        if (page >= 0) {
                            const float *mean = summaries + (int64_t(cache_page(c, b, page)) * c.kv_heads + h) * D;
#pragma unroll
                            for (int i = 0; i < D / 32; ++i) {
                                const int d = 32 * i + 4 * (lane & 7);
                                const float4 m = __ldg(reinterpret_cast<const float4 *>(mean + d));
                                double x[4];
                                q_sum(r, d, x);
                                s = fma(x[0], double(m.x), s);
                                s = fma(x[1], double(m.y), s);
                                s = fma(x[2], double(m.z), s);
                                s = fma(x[3], double(m.w), s);
                            }
                        }
#pragma unroll
                        for (int m = 4; m; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
                        return score_key(s);
                    };
                    if (doubts <= 32) { // a lane each, in the pages' order
                        uint64_t mine = 0;
                        int32_t page = -1, got = 0;
                        for (int32_t p0 = 0; p0 < most && got < doubts; p0 += 32) {
                            const uint32_t x = p0 + lane < most ? key32[p0 + lane] : 0;
                            const bool doubt = x >= cut && x <= above;
                            for (uint32_t left = __ballot_sync(0xffffffffu, doubt); left; left &= left - 1, ++got)
                                if (lane == got) page = p0 + __ffs(left) - 1;
                        }
                        for (int32_t j = 0; j < doubts; j += 4) {
                            const int32_t at = __shfl_sync(0xffffffffu, page, (j + (lane >> 3)) & 31);
                            const uint64_t y = __shfl_sync(0xffffffffu, score(at), 8 * (lane & 3));
                            if (lane >= j && lane < j + 4) mine = y;
                        }
                        int32_t rank = 0;
                        for (int32_t j = 0; j < doubts; ++j) {
                            const uint64_t y = __shfl_sync(0xffffffffu, mine, j);
                            rank += y > mine || (y == mine && j < lane);
                        }
                        if (lane < doubts) key32[page] = rank < topk - sure ? ~0u : 0;
                        __syncwarp();
                        write_bits(key32, most, above + 1, most, dst, words);
                        return;
                    }
                    // more: their scores' keys in place of the float32 ones, the largest for those above and
                    // 0 for those below. From the last pages down, since a 64-bit key covers two of the others.
                    for (int32_t p0 = (most - 1) / 32 * 32; p0 >= 0; p0 -= 32) {
                        const int32_t p = p0 + lane;
                        const uint32_t x = p < most ? key32[p] : 0;
                        uint64_t y = x > above ? ~uint64_t(0) : 0;
                        uint32_t doubt = __ballot_sync(0xffffffffu, x >= cut && x <= above);
                        while (doubt) {
                            int32_t mine = -1; // this lane's four pages' first, second, ... by its eight
                            uint32_t now = 0;
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                if (!doubt) break;
                                if (lane >> 3 == i) mine = p0 + __ffs(doubt) - 1;
                                now |= doubt & -doubt;
                                doubt &= doubt - 1;
                            }
                            const uint64_t z = __shfl_sync(0xffffffffu, score(mine),
                                                           8 * (__popc(now & ((1u << lane) - 1)) & 3));
                            if ((now >> lane) & 1u) y = z;
                        }
                        __syncwarp();
                        if (p < most) key64[p] = y;
                        __syncwarp();
                    }
                    const Keys<uint64_t, 0> e(key64, most);
                    int32_t count = e.count(1), equal = topk;
                    uint64_t edge = 1;
                    if (count > topk) {
                        edge = e.edge(topk, count);
                        if (count != topk) equal = edge == ~uint64_t(0) ? topk : topk - e.count(edge + 1);
                    }
                    write_bits(key64, most, edge, equal, dst, words);
                    return;
                }
            }
        }
        write_bits(key32, most, cut, most, dst, words);
    };
    for (int32_t r = warp; r < kRows && t0 + r < n; r += kWarps) {
        if (most <= 128) choose(r, std::integral_constant<int, 4>{});
        else if (most <= 512) choose(r, std::integral_constant<int, 16>{});
        else choose(r, std::integral_constant<int, 0>{});
    }
}

namespace {

template <int D, int kRows>
cudaError_t launch_select(const CacheView &c, const CacheQuery &q, const float *summaries, int32_t topk,
                          uint32_t *page_mask, cudaStream_t stream)
{
    auto kern = cache_select_kernel<D, kRows>;
    const size_t smem = size_t(kRows) * c.max_pages * 8; // (eight rows: max_pages <= kSelectMaxPages / 8)
    if (smem > 43 * 1024) { // (beside up to 5 KB of static shared memory)
        // the most that any call needs: a limit of this call's own would be taken from one that another
        // thread is about to launch
        const cudaError_t e =
            cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSelectMaxPages) * 8);
        if (e != cudaSuccess) return e;
    }
    const dim3 grid(kRows > 1 ? q.rows / kRows + c.batch : q.rows, c.kv_heads);
    kern<<<grid, select_warps(kRows) * 32, smem, stream>>>(c, q, summaries, topk, page_mask);
    return cudaGetLastError();
}

} // namespace

cudaError_t launch_cache_select(const CacheView &c, const CacheQuery &q, const float *summaries, int32_t topk,
                                uint32_t *page_mask, cudaStream_t stream)
{
    // Eight rows a block read each mean once; single events go one row a block. (us, 8 heads of 128,
    // one row a block and eight: 64 histories of 64 full pages, one event 9.4 and 12.8, two rows 13.9 and
    // 13.1, four 22.7 and 13.5; of 512 pages 37 and 45, 56 and 47, 100 and 51; 8 histories of 2000 pages
    // 65 and 53, 68 and 57, 72 and 56.) Rows whose eight key arrays would not fit in shared memory have to
    // go one by one, and read each mean again: 8 trees of 40 rows over 2047 pages 175, over 2065 407.
    const bool eight = q.rows > c.batch && c.max_pages <= kSelectMaxPages / 8;
    if (c.head_dim == 64)
        return eight ? launch_select<64, 8>(c, q, summaries, topk, page_mask, stream)
                     : launch_select<64, 1>(c, q, summaries, topk, page_mask, stream);
    return eight ? launch_select<128, 8>(c, q, summaries, topk, page_mask, stream)
                 : launch_select<128, 1>(c, q, summaries, topk, page_mask, stream);
}

} // namespace ba
