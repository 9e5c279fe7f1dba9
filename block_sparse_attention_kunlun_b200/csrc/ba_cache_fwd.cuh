// What the three attention kernels over the history cache (ba_cache_fwd.cu: one query row,
// CUDA cores; ba_cache_fwd_warp.cu: 8 or 16, warp-wide MMAs; ba_cache_fwd_sm100.cu: 128,
// tcgen05) share: a block's tile of query rows and which slots a row sees.
#pragma once

#include "ba_cache.cuh"

namespace ba {

// One block's work.
struct FwdTile {
    int32_t b, q0, n;       // sequence, its first row, its rows
    int32_t len;            // cached slots
    int32_t row0, rows;     // first row (token * group + head) of the tile, valid rows
    int32_t end;            // slots at and past it are empty
};

// Tile `number` of `tile_rows` rows; false: the number is unused. Warp-collective.
__device__ __forceinline__ bool find_tile(const CacheFwd &p, int64_t number, int32_t tile_rows, FwdTile &t)
{
    const int lane = threadIdx.x & 31;
    const int32_t *offs = p.q.q_offsets;
    int32_t lo = 0, n = p.c.batch;
    while (n > 1) {
        const int32_t step = (n + 31) / 32, at = lo + lane * step;
        const bool ok = lane * step < n &&
                        int64_t(__ldg(offs + at)) * p.q.group / tile_rows + (tile_rows > 1 ? at : 0) <= number;
        const int32_t cnt = __popc(__ballot_sync(0xffffffffu, ok));
        n = min(step, n - (cnt - 1) * step);
        lo += (cnt - 1) * step;
    }
    t.b = lo;
    t.q0 = __ldg(offs + lo);
    t.n = __ldg(offs + lo + 1) - t.q0;
    const int64_t first = int64_t(t.q0) * p.q.group / tile_rows + (tile_rows > 1 ? lo : 0);
    const int64_t row0 = (number - first) * tile_rows, all = int64_t(t.n) * p.q.group;
    if (row0 >= all) return false;
    t.row0 = int32_t(row0);
    t.rows = int32_t(min(all - row0, int64_t(tile_rows)));
    const int64_t cap = int64_t(p.c.max_pages) << p.c.page_shift;
    const int64_t len = max(__ldg(p.q.lens + lo), 0);
    if (len + t.n > cap && lane == 0) cache_range_error(p.c);
    t.len = int32_t(min(len, cap));
    t.end = int32_t(min(len + t.n, cap));
    return true;
}

// One query row's view of the slots.
struct RowView {
    int32_t tok, pos, ws; // token within the sequence; for pos < 0 nothing is visible: ws past every slot
};

__device__ __forceinline__ RowView row_view(const CacheFwd &p, const FwdTile &t, int32_t row)
{
    RowView r;
    r.tok = row / p.q.group;
    r.pos = query_position(p.q, t.q0, t.len, r.tok);
    r.ws = r.pos >= 0 ? rule_start(p.q, r.pos) : INT32_MAX;
    return r;
}

// First slot that rows whose windows start at `ws` or later may see: any page may be selected, and the
// rows' own slots come after the cached ones even where their positions (and windows) lie past the
// cache's last slot.
__device__ __forceinline__ int32_t first_slot(const CacheFwd &p, const FwdTile &t, int32_t ws)
{
    return p.page_mask ? 0 : min(ws, t.len);
}

// Whether row r sees slot s (s < t.end).
__device__ __forceinline__ bool sees(const CacheFwd &p, const FwdTile &t, const RowView &r, int32_t h, int32_t s)
{
    if (s < t.len) {
        if (s > r.pos) return false;
        if (s >= r.ws) return true;
        if (!p.page_mask) return false;
        const int32_t page = s >> p.c.page_shift;
        return (__ldg(p.page_mask + ((int64_t(t.q0) + r.tok) * p.c.kv_heads + h) * p.mask_words + (page >> 5)) >>
                (page & 31)) & 1u;
    }
    const int32_t j = s - t.len;
    const int32_t pj = query_position(p.q, t.q0, t.len, j);
    if (pj > r.pos || pj < r.ws) return false;
    if (!p.tree) return j <= r.tok;
    return (j >> 5) < p.tree_words &&
           ((__ldg(p.tree + (int64_t(t.q0) + r.tok) * p.tree_words + (j >> 5)) >> (j & 31)) & 1u);
}

// Stores of one finished (or, with several splits, partial) row: where it goes.
__device__ __forceinline__ int64_t out_row(const CacheFwd &p, const FwdTile &t, int32_t h, int32_t row)
{
    const int64_t token = int64_t(t.q0) + row / p.q.group;
    return token * p.c.kv_heads * p.q.group + h * p.q.group + row % p.q.group;
}

// The kernels for few rows take 16 consecutive aligned slots, always of one page, at a time.
constexpr int kGroup = 16;

// The tensor-core kernel: plan.tile_rows == kMmaRows.
constexpr int kMmaRows = 128;
template <int D>
cudaError_t launch_cache_fwd_mma(const CacheFwd &p, const CacheFwdPlan &plan, cudaStream_t stream);

// The kernel for 2 to 16 rows: plan.tile_rows 8 or 16.
template <int D>
cudaError_t launch_cache_fwd_warp(const CacheFwd &p, const CacheFwdPlan &plan, cudaStream_t stream);

// Units (pages, or halves of 128-slot pages) whose numbers a block of the tensor-core kernel
// can list: with selected pages a split covers no more slots than that.
constexpr int kMmaList = 2048;

} // namespace ba
