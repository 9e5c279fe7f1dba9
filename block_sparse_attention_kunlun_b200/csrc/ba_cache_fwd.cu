// Attention of new queries over a history cache (single events, chunks, trees of drafted
// events, candidates): block attention's serving form.
//
// Query row t of sequence b (position pos, first position its window shows ws, by the block
// rule of ba_common.cuh) sees
//   cached slot p < len        <=>  p <= pos and (p >= ws or the bit of p's page is set)
//   drafted row j (slot len+j) <=>  its tree bit is set (no tree: j <= t) and ws <= pos_j <= pos
// and out = softmax(q k / sqrt(D)) v over what it sees, lse the log of the normaliser. A row
// that sees nothing gets out = 0, lse = -inf.
//
// A block takes one tile of query rows (tokens times the heads that share a key/value head)
// and one stretch of slots (a split); with several splits the blocks leave their running
// maximum, sum and unnormalised output in float32 and cache_combine_kernel joins them in the
// order of the splits. Blocks find their sequence themselves: tiles are numbered
// floor(offs[b] * group / tile_rows) + b, which leaves at least ceil(rows / tile_rows) numbers
// for every sequence (tiles of one row simply by their row), so no pass over the batch comes
// first.
#include "ba_cache_fwd.cuh"
#include "ba_kernels.cuh"
#include "ba_ptx.cuh"

namespace ba {

namespace {

constexpr int kSimtWarps = 4; // 128 threads: one a column at the end
// blocks of the one-row kernel that an SM holds
__host__ __device__ constexpr int simt_blocks(int head_dim) { return head_dim == 128 ? 5 : 7; }

} // namespace

// One query row of one key/value head, on the CUDA cores: with one row a key, the bytes of the
// cache are the bound and even a warp-wide matrix instruction would be all but empty.
// A warp reads 16 slots of keys and of values, each a contiguous piece of its page, 16 bytes
// (16 codes) a lane: D / 16 lanes hold a slot. They are widened to float32 in registers, a
// score is a 16-term dot product in each lane and three (two) shuffles, and the value's lane
// adds its 16 columns into its own running sum: each set of D / 16 lanes keeps the running
// maximum and sum of the slots it has met, so the softmax needs no exchange inside the loop.
// The sets and the warps are joined once at the end.
// Values are on their way while scores are formed, the next slots' keys while values are added.
// One event over the windows of 256 histories (8 heads of 128, up to 512 slots each, 0.20 GB):
// 47 us, 4.3 TB/s (44 within a captured step), of which some 4 us go to the launch and, in each of a
// block's rounds, 2 to 3 to finding its sequence and pages before the first keys are under way; over
// windows of 4096 slots, whole histories mostly (1.1 GB), 213 us, and over 4096 slots of each (2.2 GB)
// 348, 6.4 TB/s. With 32 selected pages of 64 for each of 16 long histories (0.08 GB) 31 us: a split is
// a stretch of slots, whatever pages in it are selected. Five blocks an SM (four, without a bound on
// registers: 50 and 228 us where five took 47 and 223; six or seven spill: 61 and 300); at D = 64, with
// half the codes a lane, seven (30 to 32 us; five 35).
// Splitting the windows further (two, three parts) takes 12% and 21% more.
template <int D>
__global__ void __launch_bounds__(kSimtWarps * 32, simt_blocks(D)) cache_fwd_simt_kernel(const CacheFwd p)
{
    constexpr int kLanes = D / 16;      // lanes of a slot
    constexpr int kSets = 32 / kLanes;  // slots of a load
    constexpr int kU = kGroup / kSets;  // loads of a group
    __shared__ float sm_o[kSimtWarps][D];
    __shared__ float2 sm_ml[kSimtWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int32_t h = blockIdx.y, split = blockIdx.z;
    FwdTile t;
    if (!find_tile(p, blockIdx.x, 1, t)) return;
    const int col = lane % kLanes, set = lane / kLanes;
    const RowView rv = row_view(p, t, t.row0);
    const int64_t oh = out_row(p, t, h, t.row0); // the row of q and out
    float2 q[8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint4 w = __ldg(reinterpret_cast<const uint4 *>(p.q.q + oh * D + col * 16) + i);
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int x = 0; x < 4; ++x)
            q[4 * i + x] = make_float2(__uint_as_float(ws[x] << 16) * p.scale_log2,
                                       __uint_as_float(ws[x] & 0xffff0000u) * p.scale_log2);
    }
    // this split's slots, in groups of 16
    const int32_t lo = first_slot(p, t, rv.ws) / kGroup * kGroup;
    int64_t from = lo + int64_t(split) * p.chunk, to = split + 1 == p.nsplit ? t.end : from + p.chunk;
    if (to > t.end) to = t.end;
    // `from` is a multiple of 16; a split that starts past the end has nothing
    const int32_t g1 = int32_t((to + kGroup - 1) / kGroup), g0 = from < t.end ? int32_t(from / kGroup) : g1;

    float m = -INFINITY, l = 0.f;
    float2 o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = make_float2(0.f, 0.f);

    // walk of this warp's groups: 32 at a time are tested for being wanted
    int32_t base = g0 - kSimtWarps * 32, id = -1;
    uint32_t todo = 0;
    auto next_group = [&](int32_t &slot, int64_t &row) -> bool {
        while (!todo) {
            base += kSimtWarps * 32;
            if (base >= g1) return false;
            const int32_t g = base + lane * kSimtWarps + warp, s0 = g * kGroup;
            bool want = g < g1 && (s0 + kGroup > rv.ws || s0 + kGroup > t.len);
            if (g < g1 && !want && p.page_mask) {
                const int32_t page = s0 >> p.c.page_shift;
                want = (__ldg(p.page_mask + ((int64_t(t.q0) + rv.tok) * p.c.kv_heads + h) * p.mask_words +
                              (page >> 5)) >>
                        (page & 31)) & 1u;
            }
            want = want && (s0 <= rv.pos || s0 + kGroup > t.len);
            id = -1;
            if (want) {
                id = cache_page(p.c, t.b, s0 >> p.c.page_shift);
                if (id < 0) cache_range_error(p.c);
            }
            todo = __ballot_sync(0xffffffffu, id >= 0);
        }
        const int x = __ffs(todo) - 1;
        todo &= todo - 1;
        slot = (base + x * kSimtWarps + warp) * kGroup;
        row = cache_row(p.c, __shfl_sync(0xffffffffu, id, x), h, slot & ((1 << p.c.page_shift) - 1));
        return true;
    };
    // a group's codes and scale codes of keys or values
    auto load = [&](const uint8_t *codes, const uint8_t *scales, int64_t row, uint4 (&w)[kU], uint32_t (&c)[kU]) {
        const uint4 *const src = reinterpret_cast<const uint4 *>(codes + row * D) + lane;
        const uint8_t *const sc = scales + (row + set) * (D / 32) + col / 2;
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            w[u] = __ldg(src + u * 32);
            c[u] = __ldg(sc + u * kSets * (D / 32));
        }
    };

    uint4 kw[kU], vw[kU];
    uint32_t kc[kU], vc[kU];
    int32_t next_slot;
    int64_t next_row;
    bool more = next_group(next_slot, next_row);
    if (more) load(p.c.k, p.c.k_scales, next_row, kw, kc);
    while (more) {
        const int32_t slot = next_slot;
        load(p.c.v, p.c.v_scales, next_row, vw, vc);
        float s[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const uint32_t ws[4] = {kw[u].x, kw[u].y, kw[u].z, kw[u].w};
            float2 acc = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                acc = ffma2(q[i], e4m3x2_to_f32((ws[i / 2] >> (16 * (i % 2))) & 0xffffu), acc);
            s[u] = (acc.x + acc.y) * mx_scale(kc[u]);
        }
        more = next_group(next_slot, next_row);
        if (more) load(p.c.k, p.c.k_scales, next_row, kw, kc);
        // the slots that the row sees
        uint32_t vis = 0xffffu;
        if (!(slot >= rv.ws && slot + kGroup - 1 <= min(rv.pos, t.len - 1)))
            vis = __ballot_sync(0xffffffffu, lane < kGroup && slot + lane < t.end && sees(p, t, rv, h, slot + lane));
        float mx = m;
#pragma unroll
        for (int u = 0; u < kU; ++u) {
#pragma unroll
            for (int x = 1; x < kLanes; x <<= 1) s[u] += __shfl_xor_sync(0xffffffffu, s[u], x);
            s[u] = (vis >> (u * kSets + set)) & 1u ? s[u] : -INFINITY;
            mx = fmaxf(mx, s[u]);
        }
        const float ref = mx == -INFINITY ? 0.f : mx;
        const float alpha = ex2_approx(m - ref);
        m = mx;
        float sum = 0.f;
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            s[u] = ex2_approx(s[u] - ref);
            sum += s[u];
        }
        l = fmaf(l, alpha, sum);
        if (__any_sync(0xffffffffu, alpha != 1.f)) {
            const float2 a2 = make_float2(alpha, alpha);
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = fmul2(o[i], a2);
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            // a slot that the row does not see may hold anything (0 * NaN is NaN)
            if (!((vis >> (u * kSets + set)) & 1u)) continue;
            const uint32_t ws[4] = {vw[u].x, vw[u].y, vw[u].z, vw[u].w};
            const float pr = s[u] * mx_scale(vc[u]);
            const float2 pr2 = make_float2(pr, pr);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                o[i] = ffma2(pr2, e4m3x2_to_f32((ws[i / 2] >> (16 * (i % 2))) & 0xffffu), o[i]);
        }
    }

    // join the sets of lanes, then the warps
    float mx = m;
#pragma unroll
    for (int x = kLanes; x < 32; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
    const float a = ex2_approx(m - (mx == -INFINITY ? 0.f : mx));
    l *= a;
#pragma unroll
    for (int x = kLanes; x < 32; x <<= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        o[i].x *= a;
        o[i].y *= a;
#pragma unroll
        for (int x = kLanes; x < 32; x <<= 1) {
            o[i].x += __shfl_xor_sync(0xffffffffu, o[i].x, x);
            o[i].y += __shfl_xor_sync(0xffffffffu, o[i].y, x);
        }
    }
    if (set == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) *reinterpret_cast<float2 *>(&sm_o[warp][col * 16 + 2 * i]) = o[i];
    }
    if (lane == 0) sm_ml[warp] = make_float2(mx, l);
    __syncthreads();
    const int32_t d = threadIdx.x;
    if (d >= D) return;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kSimtWarps; ++w) top = fmaxf(top, sm_ml[w].x);
    const float ref = top == -INFINITY ? 0.f : top;
    float sum = 0.f, acc = 0.f;
#pragma unroll
    for (int w = 0; w < kSimtWarps; ++w) {
        const float x = ex2_approx(sm_ml[w].x - ref);
        sum = fmaf(sm_ml[w].y, x, sum);
        acc = fmaf(sm_o[w][d], x, acc);
    }
    const int32_t heads = p.c.kv_heads * p.q.group;
    if (p.nsplit == 1) {
        p.out[oh * D + d] = __float2bfloat16(sum == 0.f ? 0.f : acc / sum);
        if (d == 0) p.lse[oh % heads * p.q.rows + oh / heads] = (top + log2f(sum)) * 0.6931471805599453f;
    } else {
        const int64_t at = int64_t(split) * p.q.rows * heads + oh;
        p.part_o[at * D + d] = acc;
        if (d == 0) p.part_ml[at] = make_float2(top, sum);
    }
}

// Joins the splits of every (row, head): weights 2^(m_s - max m), in the order of the splits.
// One warp per row and head, D / 32 columns a lane; bound by its launch and the latency of
// its reads (some 5 us of the 113 to 116 of 16 candidate sets in four splits).
template <int D>
__global__ void __launch_bounds__(256) cache_combine_kernel(const CacheFwd p)
{
    constexpr int C = D / 32;
    const int lane = threadIdx.x & 31;
    const int32_t heads = p.c.kv_heads * p.q.group;
    const int64_t all = int64_t(p.q.rows) * heads, at = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (at >= all || at / heads >= __ldg(p.q.q_offsets + p.c.batch)) return; // (rows behind the last sequence)
    float mx = -INFINITY;
    for (int32_t s = 0; s < p.nsplit; ++s) mx = fmaxf(mx, p.part_ml[s * all + at].x);
    const float ref = mx == -INFINITY ? 0.f : mx;
    float sum = 0.f, acc[C];
#pragma unroll
    for (int i = 0; i < C; ++i) acc[i] = 0.f;
    for (int32_t s = 0; s < p.nsplit; ++s) {
        const float2 ml = p.part_ml[s * all + at];
        if (ml.x == -INFINITY && ml.y == 0.f) continue; // nothing seen there
        const float a = ex2_approx(ml.x - ref);
        sum = fmaf(ml.y, a, sum);
        const float *src = p.part_o + (s * all + at) * D + lane * C;
#pragma unroll
        for (int i = 0; i < C; ++i) acc[i] = fmaf(src[i], a, acc[i]);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int i = 0; i < C; i += 2)
        *reinterpret_cast<uint32_t *>(p.out + at * D + lane * C + i) = pack_bf16x2(acc[i] * inv, acc[i + 1] * inv);
    if (lane == 0) {
        const int64_t token = at / heads, head = at % heads;
        p.lse[head * p.q.rows + token] = (mx + log2f(sum)) * 0.6931471805599453f;
    }
}

CacheFwdPlan cache_fwd_plan(int32_t batch, int32_t rows, int32_t kv_heads, int32_t group, int32_t head_dim,
                            int64_t slots, int32_t page_size, int64_t block, int64_t window,
                            bool has_mask)
{
    CacheFwdPlan plan;
    const int64_t all = int64_t(rows) * group; // query rows of a key/value head
    // sequences that can have rows: a batch padded with empty ones is planned as the rest of it, and no
    // sequence counts for less than the rows that one token brings
    const int64_t live = batch < rows ? batch : rows;
    const int64_t each = live > 0 ? (all + live - 1) / live : 1;
    // The kernel goes by the rows of a sequence on average. (us for tiles of 8, 16, 128 rows, trees of so many
    // rows. 64 windows of four 512: 8 rows 71, 103, 114; 12 124, 105, 115; 16 123, 109, 116; 17 -, 165, 117;
    // 32 -, 176, 121. 8 whole histories of 16,000 to 33,000: 8 rows 122, 159, 191; 12 196, 161, 192; 16 200,
    // 162, 192; 17 -, 255, 192; 32 -, 270, 195. One event, 16 whole histories of 25,000 to 33,000, on the
    // CUDA cores, 8, 16: one head 163, 227, 296; two 287, 224, 297; four 546, 222, 296.) A batch of unlike
    // sequences pays for that: 255 single events over windows take 44 us and a chunk of 512 rows 21, together,
    // in tiles of 8 rows, 87 (under four heads 63, 33 and, in tiles of 16, 169).
    plan.tile_rows = each <= 1 ? 1 : (each <= 8 ? 8 : (each <= 16 ? 16 : kMmaRows));
    const bool mma = plan.tile_rows == kMmaRows;
    plan.tiles = plan.tile_rows > 1 ? all / plan.tile_rows + batch : all;
    // the most slots a tile may meet: the whole cache, or the window and the rows themselves
    int64_t reach = slots;
    if (!has_mask) {
        const int64_t per = live > 0 ? (int64_t(rows) + live - 1) / live : 0;
        if (window < slots && block < slots && block * window + per < slots) reach = block * window + per;
    }
    // Splits: as many as fill the blocks that a B200's 148 SMs hold at once (a constant: the workspace query
    // must say the same without a device), or three times that (twice on the tensor cores) where a split
    // still has 1024 slots, none of fewer than 256. With more items than places nothing is split, and
    // the last round of blocks is as full as it happens to be. (us for three rounds, two, one. One event
    // over 16 histories of 25,000 to 33,000: four heads 215, 222, 256, sixteen 309, 333, 349, one 166, 172, 197;
    // over two, four heads, 43 each. On the tensor cores, where no one of them is best: 16 candidate sets with
    // selected pages 115, 109, 118; 8 trees over whole histories 194, 182, 195; 32 of 64 rows over 8192 slots
    // 263, 252, 230; 16 chunks of 128 to 512 rows over windows 143, 117, 117; one of 512 over 32,768 slots
    // 166, 145, 130; 8 or 64 trees over windows, in splits of fewer slots or none, alike.)
    const int64_t held = 148 * (mma ? 2 : plan.tile_rows == 1 ? simt_blocks(head_dim) : plan.tile_rows == 8 ? 4 : 3);
    const int64_t work = (all + plan.tile_rows - 1) / plan.tile_rows;
    const int64_t items = (work > live ? work : live) * kv_heads;
    int64_t n = items > 0 ? (mma ? 2 : 3) * held / items : 1;
    if (n > 1 && reach / n < 1024) n = held / items;
    const int64_t most = (reach + 255) / 256;
    if (n > most) n = most;
    if (n < 1) n = 1;
    int64_t chunk = ((reach + n - 1) / n + 63) / 64 * 64;
    if (mma && has_mask) {
        const int64_t unit = page_size < 64 ? page_size : 64;
        if (chunk > kMmaList * unit) chunk = kMmaList * unit;
    }
    plan.chunk = int32_t(chunk);
    plan.nsplit = int32_t((reach + chunk - 1) / chunk);
    if (plan.nsplit < 1) plan.nsplit = 1;
    const size_t parts = plan.nsplit > 1 ? size_t(plan.nsplit) * size_t(all) * kv_heads : 0;
    plan.bytes = align256(parts * 8) + align256(parts * head_dim * 4);
    return plan;
}

namespace {

template <int D>
cudaError_t launch_d(const CacheFwd &p, const CacheFwdPlan &plan, cudaStream_t stream)
{
    if (plan.tile_rows == kMmaRows) {
        const cudaError_t e = launch_cache_fwd_mma<D>(p, plan, stream);
        if (e != cudaSuccess) return e;
    } else if (plan.tile_rows > 1) {
        const cudaError_t e = launch_cache_fwd_warp<D>(p, plan, stream);
        if (e != cudaSuccess) return e;
    } else {
        const dim3 grid(unsigned(plan.tiles), unsigned(p.c.kv_heads), unsigned(p.nsplit));
        cache_fwd_simt_kernel<D><<<grid, kSimtWarps * 32, 0, stream>>>(p);
    }
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || p.nsplit == 1) return e;
    const int64_t rows = int64_t(p.q.rows) * p.c.kv_heads * p.q.group;
    cache_combine_kernel<D><<<unsigned((rows + 7) / 8), 256, 0, stream>>>(p);
    return cudaGetLastError();
}

} // namespace

cudaError_t launch_cache_fwd(const CacheFwd &p, const CacheFwdPlan &plan, cudaStream_t stream)
{
    return p.c.head_dim == 64 ? launch_d<64>(p, plan, stream) : launch_d<128>(p, plan, stream);
}

} // namespace ba
