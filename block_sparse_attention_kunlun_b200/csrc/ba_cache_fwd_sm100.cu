// Attention over the history cache on the tensor cores: up to 128 query rows (tokens times
// the heads that share a key/value head) of one sequence against 64 slots at a time. The
// rule, the tiles and the splits are ba_cache_fwd.cu's.
//
// S = Q K^T and O += P V run as tcgen05 MMAs (M = 128 rows, bf16 operands, float32
// accumulators in TMEM) whose A operands, Q and P, stay in TMEM: shared memory then carries
// only keys and values. Those are MX codes in the cache. A head's slots of a page are
// consecutive, so bulk copies bring codes and scales of 64 slots into shared memory with no
// registers held meanwhile (loads into registers, one tile ahead, left the dequantising warps
// waiting: 3200 cycles a tile); the dequantising warps widen them to bf16 (exact: an E4M3
// value has four significant bits and the scale is a power of two) and store them in the
// MMA's 128-byte-swizzled layout. A tensor product on the codes themselves would have to round Q
// to E4M3, and the values' scales run along head_dim, not along the keys that P V sums over.
// P is rounded to bf16 for its MMA, as in ba_fwd; the running sum takes the unrounded probabilities. (out is
// then off by 0.0019 of its size, root mean square, where its own rounding makes 0.0016. P in two bf16 parts
// would end at 0.0016, with twice the MMAs of P V: 140 us for the trees below, 123 for the candidates.)
//
// Roles of a block (512 threads, two blocks an SM, so that one block's softmax and set-up
// overlap the other's MMAs):
//   warps 0-3   softmax: thread t owns row t (TMEM lane t)
//   warps 4-11  dequantisation of a 64-slot tile
//   warp 14     bulk copies of the tiles' codes
//   warp 15     MMA issue (on another scheduler than the first softmax warps; 12 and 13 only
//               fill the warpgroup, whose registers go to the softmax)
// TMEM columns: O at 0, S at 128 (P over its first 32), Q at 192.
//
// Columns are kept in the order that widening four codes at once gives, 0 2 1 3 within each
// four: Q is put in the same order as it is loaded, O is put back as it is stored.
//
// 64 trees of 5 to 64 rows over windows of four blocks of 512 (8 heads of 128, 0.25 GB): 124 to 126 us;
// 16 sets of 33 to 64 candidates with 32 selected pages a row (group of two, 0.12 GB): 113 to 116 us;
// 16 chunks of 512 rows over such windows: 143 us, 420 TFLOP/s.
// Not bytes but the chain of a tile bounds it, which the two blocks of an SM overlap by half.
// Clocked in the first case, in cycles: S's eight MMAs take 340 to issue and 330 more to finish,
// S's load 260, the maximum 130, the exponentials 710, storing P 135, the hand-over 90, P V's MMAs
// 410: 2450 at best, 3000 with the other block in the way; widening is a tile ahead. The MMAs take
// their 750 however few of the 128 rows there are. Without the widening's and the exponentials'
// arithmetic the first case would take 106 us, without the MMAs too 86; a block's set-up (sequence,
// Q, page list, TMEM) is 16 of them in the first case and 30 in the second. S in halves of 32
// slots, one ahead of the softmax, took 133 us (more and narrower MMAs), codes by loads into
// registers 179, one block an SM with all roles doubled 270, codes brought into L2 three tiles
// ahead 130.
//
// With selected pages the block first lists the units (pages, or halves of 128-slot pages)
// that any of its rows sees, so that small pages far apart share a tile.
#include "ba_cache_fwd.cuh"
#include "ba_kernels.cuh"
#include "ba_ptx.cuh"

#include <type_traits>

namespace ba {

namespace {

// Copy of `bytes` consecutive bytes into shared memory, completing on `bar`; both addresses
// and the size must be multiples of 16.
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

constexpr int kKeys = 64; // slots of a tile
constexpr int kThreads = 512;
constexpr int kCopyWarp = 14, kMmaWarp = 15;
// registers a thread after the split (softmax, dequantisation, MMA warpgroup); two blocks of
// 512 threads are launched with 64 each: 104 + 2 * 56 + 40 = 4 * 64
constexpr uint32_t kRegsSoftmax = 104, kRegsDequant = 56, kRegsMma = 40;

template <int D>
struct MmaLayout {
    static_assert(D == 64 || D == 128, "head_dim 64 or 128");
    // stages of widened tiles (K, then V) and of codes (K, V, K scales, V scales): 97 KB for
    // either D, so that two blocks fit an SM and never three, whose TMEM (256 columns each) would not
    static constexpr int kStages = D == 128 ? 2 : 4, kRawStages = kStages;
    static constexpr int kChunkBytes = kKeys * 128;      // 64 slots x 64 columns, bf16
    static constexpr int kTileBytes = kKeys * D * 2;
    static constexpr int kRaw0 = 2 * kStages * kTileBytes;
    static constexpr int kRawV = kKeys * D, kRawKs = 2 * kRawV, kRawVs = kRawKs + kRawV / 32;
    static constexpr int kRawBytes = 2 * kRawV + 2 * kRawV / 32;
    static constexpr int kBytes = kRaw0 + kRawStages * kRawBytes;
    static constexpr int kAlloc = kBytes + 1024;
    static constexpr uint32_t kTmemCols = 256, kColO = 0, kColS = 128, kColQ = 192;
};

struct MmaShared {
    uint64_t full[4], empty[4];         // stages of widened K and V
    uint64_t raw_full[4], raw_empty[4]; // stages of codes
    // per tile (mod 16, more than can be under way): how many slots of each 16 there are, a byte each
    uint32_t there[16];
    uint64_t s_full, p_full, o_final;
    uint32_t tmem;
    int abort;
    int32_t min_ws, max_pos; // over the tile's rows
    int32_t nlist;
    int32_t odd_values;      // some value is NaN or infinite
    int32_t holes;           // some page has no number
    uint32_t wanted[kMmaList / 32 + 1];
    int32_t list[kMmaList];  // first slots of the listed units
};

// What a block's roles know of its slots.
struct Slots {
    int32_t first;   // slots before it are seen by no row
    int32_t from;    // first slot of the split (no list)
    int32_t shift;   // log2 of a unit's slots (no list: the whole tile is one)
    int32_t end;     // slots at and past it do not exist
    int32_t ntiles;
    bool listed;
};

// First slot of unit k of tile i; past the list: INT32_MAX - 63.
__device__ __forceinline__ int32_t unit_slot(const Slots &s, const MmaShared &sb, int32_t i, int32_t k)
{
    if (!s.listed) return s.from + i * kKeys + (k << s.shift);
    const int32_t x = i * (kKeys >> s.shift) + k;
    return x < sb.nlist ? sb.list[x] : INT32_MAX - 63;
}

// Bits lo .. hi (clamped to 0 .. n - 1) of a 64-bit word.
__device__ __forceinline__ uint64_t bit_range(int64_t lo, int64_t hi, int32_t n)
{
    if (lo < 0) lo = 0;
    if (hi > n - 1) hi = n - 1;
    return lo <= hi ? (~uint64_t(0) >> (63 - hi)) & (~uint64_t(0) << lo) : 0;
}

// Which of the n slots from `us` on row r sees.
__device__ __forceinline__ uint64_t visible_bits(const CacheFwd &p, const FwdTile &t, const RowView &r, int32_t h,
                                                 int32_t us, int32_t n, int32_t end)
{
    if (us >= end) return 0;
    int32_t ws = r.ws;
    if (p.page_mask && us < t.len && us < ws) {
        const int32_t page = us >> p.c.page_shift;
        if ((__ldg(p.page_mask + ((int64_t(t.q0) + r.tok) * p.c.kv_heads + h) * p.mask_words + (page >> 5)) >>
             (page & 31)) & 1u)
            ws = 0;
    }
    uint64_t bits = bit_range(int64_t(ws) - us, int64_t(min(r.pos, t.len - 1)) - us, n);
    if (us + n > t.len) { // the unit holds drafted rows: slots first .. stop - 1
        const int32_t first = max(us, t.len), stop = min(us + n, end);
        if (!p.tree && !p.q.positions) {
            bits |= bit_range(int64_t(max(r.ws, t.len)) - us, int64_t(min(r.pos, end - 1)) - us, n);
        } else {
            // rows by the tree (or before this one), then their positions one by one
            uint64_t rows = bit_range(first - us, stop - 1 - us, n);
            if (!p.tree) {
                rows &= bit_range(0, int64_t(t.len) + r.tok - us, n);
            } else {
                uint64_t sees = 0;
                const uint32_t *words = p.tree + (int64_t(t.q0) + r.tok) * p.tree_words;
                for (int32_t w = (first - t.len) >> 5; w <= (stop - 1 - t.len) >> 5 && w < p.tree_words; ++w) {
                    const int32_t at = t.len + 32 * w - us; // the unit's bit of the word's first row
                    const uint64_t word = __ldg(words + w);
                    sees |= at >= 0 ? word << at : word >> -at;
                }
                rows &= sees;
            }
            for (uint64_t left = rows; left; left &= left - 1) {
                const int32_t x = __ffsll(int64_t(left)) - 1;
                const int32_t pj = query_position(p.q, t.q0, t.len, us + x - t.len);
                if (pj > r.pos || pj < r.ws) rows &= ~(uint64_t(1) << x);
            }
            bits |= rows;
        }
    }
    return bits;
}

// Sixteen E4M3 codes with the scale code of their block as bf16, exactly (the products
// below bf16's normal range round to its subnormals), columns in the order 0 2 1 3 within
// each four. A code's sign, exponent and mantissa moved to a bf16's places (sign to bit 15,
// the other seven bits to bits 10 .. 4) are the value times 2^-120, subnormal codes included;
// one multiplication by 2^(e + 120) makes up for that and applies the scale. Returns whether
// that holds: not for a NaN code, nor for scales past 2^7, whose factor is none of bf16's
// (widen4_any then).
__device__ __forceinline__ bool widen16(const uint4 &codes, uint32_t scale_code, uint32_t (&out)[8])
{
    const uint32_t ws[4] = {codes.x, codes.y, codes.z, codes.w};
    const uint32_t f = scale_code * 0x00800080u + 0x3c003c00u;
    const __nv_bfloat162 s = *reinterpret_cast<const __nv_bfloat162 *>(&f);
    uint32_t nan = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w = ws[i];
        nan |= (w & 0x7f7f7f7fu) + 0x01010101u; // a NaN's byte becomes 0x80
        const uint32_t x[2] = {((w << 4) & 0x07f007f0u) | ((w << 8) & 0x80008000u),
                               ((w >> 4) & 0x07f007f0u) | (w & 0x80008000u)};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&x[j]), s);
            out[2 * i + j] = *reinterpret_cast<const uint32_t *>(&v);
        }
    }
    return !(nan & 0x80808080u) && scale_code <= 134;
}

// Four codes of any kind in the same form. With clear, NaNs and infinities become 0 and *odd
// says that there were any. (Out of line and rare; its arguments are values, so that the
// registers of the common path stay registers.)
__device__ __noinline__ uint2 widen4_any(uint32_t codes, uint32_t scale_code, bool clear, int32_t *odd)
{
    uint32_t o[2] = {0u, 0u};
    for (int i = 0; i < 4; ++i) { // code i is in word i % 2, half i / 2
        const float f = e4m3x2_to_f32((codes >> (8 * i)) & 0xffu).x * mx_scale(scale_code);
        uint32_t v = __bfloat16_as_ushort(__float2bfloat16(f));
        if (clear && (v & 0x7f80u) == 0x7f80u) {
            v = 0;
            *odd = 1;
        }
        o[i % 2] |= v << (16 * (i / 2));
    }
    return make_uint2(o[0], o[1]);
}

// Columns of this row's output that a NaN, +infinity or -infinity among the values it sees
// must reach. P V runs on values with those cleared, because a row that does not see them
// would multiply them by zero; the rows that do are mended here, from the codes. Called by
// whole warps, lane = row; one 4-byte word of codes a lane.
template <int D>
struct OddValues {
    uint32_t nan[D / 32], pos[D / 32], neg[D / 32];
};

template <int D>
__device__ __noinline__ void find_odd_values(const CacheFwd &p, const FwdTile &t, const RowView &r, int32_t h,
                                             const Slots &sl, const MmaShared &sb, OddValues<D> &odd)
{
    const int lane = threadIdx.x & 31;
    for (int w = 0; w < D / 32; ++w) odd.nan[w] = odd.pos[w] = odd.neg[w] = 0;
    for (int32_t i = 0; i < sl.ntiles; ++i)
        for (int32_t c = 0; c < kKeys; ++c) {
            const int32_t slot = unit_slot(sl, sb, i, c >> sl.shift) + (c & ((1 << sl.shift) - 1));
            if (slot >= sl.end) continue;
            const int32_t id = cache_page(p.c, t.b, slot >> p.c.page_shift);
            if (id < 0) continue;
            const int64_t row = cache_row(p.c, id, h, slot & ((1 << p.c.page_shift) - 1));
            uint32_t n = 0, a = 0, b = 0;
            if (lane < D / 4) {
                const uint32_t codes = __ldg(reinterpret_cast<const uint32_t *>(p.c.v + row * D) + lane);
                const float s = mx_scale(__ldg(p.c.v_scales + row * (D / 32) + lane / 8));
                for (int x = 0; x < 4; ++x) {
                    const uint32_t code = (codes >> (8 * x)) & 0xffu;
                    const float f = __bfloat162float(__float2bfloat16(e4m3x2_to_f32(code).x * s));
                    n |= uint32_t(f != f) << x;
                    a |= uint32_t(f == INFINITY) << x;
                    b |= uint32_t(f == -INFINITY) << x;
                }
            }
            if (!__any_sync(0xffffffffu, n | a | b)) continue;
            const bool mine = sees(p, t, r, h, slot);
            for (int w = 0; w < D / 32; ++w) {
                const int sh = 4 * (lane % 8);
                const bool here = lane / 8 == w;
                const uint32_t nw = __reduce_or_sync(0xffffffffu, here ? n << sh : 0u);
                const uint32_t aw = __reduce_or_sync(0xffffffffu, here ? a << sh : 0u);
                const uint32_t bw = __reduce_or_sync(0xffffffffu, here ? b << sh : 0u);
                if (mine) {
                    odd.nan[w] |= nw;
                    odd.pos[w] |= aw;
                    odd.neg[w] |= bw;
                }
            }
        }
}

} // namespace

template <int D>
__global__ void __launch_bounds__(kThreads, 2) cache_fwd_mma_kernel(const __grid_constant__ CacheFwd p)
{
    using Lay = MmaLayout<D>;
    constexpr int S = Lay::kStages;
    extern __shared__ uint8_t smem_raw[];
    __shared__ MmaShared sb;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t smem_base = smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int32_t h = blockIdx.y, split = blockIdx.z;
    FwdTile t;
    if (!find_tile(p, blockIdx.x, kMmaRows, t)) return;
    const int active = (t.rows + 31) / 32; // softmax warps with rows
    if (split > 0 && int64_t(split) * p.chunk >= t.end) { // a split past the history's end
        if (tid < t.rows)
            p.part_ml[int64_t(split) * p.q.rows * p.c.kv_heads * p.q.group + out_row(p, t, h, t.row0 + tid)] =
                make_float2(-INFINITY, 0.f);
        return;
    }

    if (tid == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&sb.full[i], 8);
            mbar_init(&sb.empty[i], 1);
            mbar_init(&sb.raw_full[i], 1);
            mbar_init(&sb.raw_empty[i], 8);
        }
        mbar_init(&sb.s_full, 1);
        mbar_init(&sb.p_full, active);
        mbar_init(&sb.o_final, 1);
        sb.abort = 0;
        sb.min_ws = INT32_MAX;
        sb.max_pos = -1;
        sb.nlist = 0;
        sb.odd_values = 0;
        sb.holes = 0;
        fence_mbar_init();
    }
    if (p.page_mask)
        for (int i = tid; i < kMmaList / 32 + 1; i += kThreads) sb.wanted[i] = 0;
    if (warp == kMmaWarp) {
        tmem_alloc(&sb.tmem, Lay::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sb.tmem;
    volatile int *abort = &sb.abort;

    const int32_t row = t.row0 + min(tid, t.rows - 1);
    const RowView rv = row_view(p, t, row); // (warps past the rows: the last row's)
    const uint32_t lane_base = uint32_t((warp & 3) * 32) << 16;
    if (warp < active) {
        const int32_t mw = __reduce_min_sync(0xffffffffu, rv.ws), mp = __reduce_max_sync(0xffffffffu, rv.pos);
        if (lane == 0) {
            atomicMin(&sb.min_ws, mw);
            atomicMax(&sb.max_pos, mp);
        }
        // this row of Q into TMEM
        const uint4 *src = reinterpret_cast<const uint4 *>(p.q.q + out_row(p, t, h, row) * D);
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
            uint32_t w[32];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const uint4 x = __ldg(src + 8 * c + u);
                w[4 * u] = __byte_perm(x.x, x.y, 0x5410), w[4 * u + 1] = __byte_perm(x.x, x.y, 0x7632);
                w[4 * u + 2] = __byte_perm(x.z, x.w, 0x5410), w[4 * u + 3] = __byte_perm(x.z, x.w, 0x7632);
            }
            tmem_st32(tmem + lane_base + Lay::kColQ + 32 * c, w);
        }
        tmem_wait_st();
    }
    __syncthreads();

    // this split's slots
    Slots sl;
    sl.listed = p.page_mask != nullptr;
    const int32_t size = 1 << p.c.page_shift;
    sl.shift = sl.listed ? min(p.c.page_shift, 6) : 6;
    const int32_t unit = 1 << sl.shift;
    sl.end = t.end;
    if (!p.tree && !p.q.positions)
        sl.end = int32_t(min(int64_t(t.end), int64_t(t.len) + (t.row0 + t.rows - 1) / p.q.group + 1));
    const int32_t min_ws = sb.min_ws;
    sl.first = first_slot(p, t, min_ws);
    const int64_t from = sl.first / kKeys * kKeys + int64_t(split) * p.chunk;
    int64_t to = split + 1 == p.nsplit ? sl.end : from + p.chunk;
    if (to > sl.end) to = sl.end;
    sl.from = int32_t(min(from, int64_t(sl.end)));
    sl.ntiles = from < to ? int32_t((to - from + kKeys - 1) / kKeys) : 0;
    if (sl.listed) {
        // bits of the pages from `from` on that a row selects, then the list of units
        const int32_t page0 = sl.from >> p.c.page_shift;
        const int32_t npages = from < to ? int32_t((to - 1) >> p.c.page_shift) - page0 + 1 : 0;
        const int32_t tok0 = t.row0 / p.q.group, ntok = (t.row0 + t.rows - 1) / p.q.group - tok0 + 1;
        const int32_t w0 = page0 >> 5, nw = npages > 0 ? ((page0 + npages - 1) >> 5) - w0 + 1 : 0;
        for (int32_t x = tid; x < nw * ntok; x += kThreads) {
            const int32_t w = x % nw, tok = tok0 + x / nw;
            const uint32_t bits = __ldg(p.page_mask + ((int64_t(t.q0) + tok) * p.c.kv_heads + h) * p.mask_words + w0 + w);
            if (bits) atomicOr(&sb.wanted[w], bits);
        }
        __syncthreads();
        if (warp == 0) {
            const int32_t nunits = from < to ? int32_t((to - from + unit - 1) >> sl.shift) : 0;
            int32_t count = 0;
            for (int32_t u0 = 0; u0 < nunits; u0 += 32) {
                const int32_t us = sl.from + ((u0 + lane) << sl.shift);
                bool want = false;
                if (u0 + lane < nunits) {
                    const int32_t page = us >> p.c.page_shift;
                    const bool bit = (sb.wanted[(page >> 5) - w0] >> (page & 31)) & 1u;
                    want = (us < t.len && us <= sb.max_pos && (bit || us + unit > min_ws)) || us + unit > t.len;
                }
                const uint32_t b = __ballot_sync(0xffffffffu, want);
                if (want) sb.list[count + __popc(b & ((1u << lane) - 1))] = us;
                count += __popc(b);
            }
            if (lane == 0) sb.nlist = count;
        }
        __syncthreads();
        const int32_t per = kKeys >> sl.shift;
        sl.ntiles = (sb.nlist + per - 1) / per;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();

    if (warp < 4) {
        warpgroup_regs_inc<kRegsSoftmax>();
        // ------------------------------------------------------ softmax ---
        if (warp < active) {
        const bool valid = tid < t.rows;
        const uint32_t s_addr = tmem + lane_base + Lay::kColS, o_addr = tmem + lane_base + Lay::kColO;
        const int32_t last = min(rv.pos, t.len - 1); // cached slots from rv.ws to here are seen
        float m_ref = -INFINITY, l = 0.f;
        bool ok = true;
        for (int32_t i = 0; i < sl.ntiles; ++i) {
            uint64_t bits = 0;
            if (!sl.listed) {
                const int32_t s0 = sl.from + i * kKeys;
                bits = s0 >= rv.ws && s0 + kKeys - 1 <= last ? ~uint64_t(0)
                                                              : visible_bits(p, t, rv, h, s0, kKeys, sl.end);
            } else {
                for (int32_t k = 0; k < kKeys >> sl.shift; ++k)
                    bits |= visible_bits(p, t, rv, h, unit_slot(sl, sb, i, k), unit, sl.end)
                            << (k << sl.shift);
            }
            if (!mbar_wait(&sb.s_full, i & 1, abort)) {
                ok = false;
                break;
            }
            tc_fence_after();
            if (*const_cast<volatile int32_t *>(&sb.holes)) { // slots whose page has no number are unseen
                const uint32_t there = sb.there[i % 16];
                for (int g = 0; g < 4; ++g)
                    if (((there >> (8 * g)) & 0xffu) == 0) bits &= ~(uint64_t(0xffff) << (16 * g));
            }
            const uint32_t vis[2] = {uint32_t(bits), uint32_t(bits >> 32)};
            const bool full = __all_sync(0xffffffffu, (vis[0] & vis[1]) == 0xffffffffu);
            uint32_t sr[2][32];
            tmem_ld32(s_addr, sr[0]);
            tmem_ld32(s_addr + 32, sr[1]);
            tmem_wait_ld();
            reg_fence(sr[0]);
            reg_fence(sr[1]);
            if (!full) {
#pragma unroll
                for (int c = 0; c < kKeys; ++c)
                    sr[c / 32][c % 32] = (vis[c / 32] & (1u << (c % 32))) ? sr[c / 32][c % 32] : 0xff800000u;
            }
            float mp[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < kKeys; c += 2)
                mp[(c / 2) % 4] = fmax3(mp[(c / 2) % 4], __uint_as_float(sr[c / 32][c % 32]),
                                        __uint_as_float(sr[c / 32][c % 32 + 1]));
            const float m_new = fmaxf(fmaxf(mp[0], mp[1]), fmaxf(mp[2], mp[3])) * p.scale_log2;
            // O and l move to the new maximum only when it grew by more than 2^8
            float alpha = 1.f;
            const bool grow = m_new > m_ref + 8.0f;
            if (grow) {
                alpha = ex2_approx(m_ref - m_new);
                m_ref = m_new;
            }
            const float neg_m = m_ref == -INFINITY ? 0.f : -m_ref;
            const float2 sc2 = make_float2(p.scale_log2, p.scale_log2), nm2 = make_float2(neg_m, neg_m);
            float2 acc[2] = {{0.f, 0.f}, {0.f, 0.f}};
            uint32_t pk[32];
#pragma unroll
            for (int c = 0; c < 32; ++c) {
                const float2 x = ffma2(make_float2(__uint_as_float(sr[c / 16][2 * (c % 16)]),
                                                   __uint_as_float(sr[c / 16][2 * (c % 16) + 1])),
                                       sc2, nm2);
                const float p0 = ex2_approx(x.x), p1 = ex2_approx(x.y);
                acc[c % 2] = fadd2(acc[c % 2], make_float2(p0, p1));
                pk[c] = pack_bf16x2(p0, p1);
            }
            tmem_st32(s_addr, pk);
            const float2 sum = fadd2(acc[0], acc[1]);
            l = fmaf(l, alpha, sum.x + sum.y);
            // O holds the earlier tiles' P V (complete: this S was issued after it)
            if (i > 0 && __any_sync(0xffffffffu, grow)) {
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    tmem_ld32(o_addr + c * 32, o);
                    tmem_wait_ld();
                    reg_fence(o);
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
                    tmem_st32(o_addr + c * 32, o);
                }
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sb.p_full);
        }
        if (ok && sl.ntiles > 0) ok = mbar_wait(&sb.o_final, 0, abort);
        if (ok) {
            tc_fence_after();
            OddValues<D> odd;
            const bool any_odd = sl.ntiles > 0 && *reinterpret_cast<volatile int32_t *>(&sb.odd_values);
            if (any_odd) { // (copies: objects whose address is taken would live in memory throughout)
                const FwdTile t2 = t;
                const RowView r2 = rv;
                const Slots s2 = sl;
                OddValues<D> o2;
                find_odd_values<D>(p, t2, r2, h, s2, sb, o2);
                odd = o2;
            }
            const int64_t oh = out_row(p, t, h, row);
            const int64_t heads = int64_t(p.c.kv_heads) * p.q.group;
            const bool whole = p.nsplit == 1;
            const int64_t at = whole ? oh : int64_t(split) * p.q.rows * heads + oh;
            const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
            // a part without any visible slot is left out by its statistics
            const bool store = valid && (whole || l != 0.f);
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                if (sl.ntiles > 0) {
                    tmem_ld32(o_addr + c * 32, o);
                    tmem_wait_ld();
                    reg_fence(o);
                } else {
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = 0;
                }
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    o[k] = l == 0.f ? 0u : __float_as_uint(__uint_as_float(o[k]) * inv);
#pragma unroll
                for (int k = 0; k < 32; k += 4) { // 0 2 1 3 back to 0 1 2 3
                    const uint32_t x = o[k + 1];
                    o[k + 1] = o[k + 2];
                    o[k + 2] = x;
                }
                if (any_odd) {
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        const uint32_t b = 1u << k;
                        const bool a = odd.pos[c] & b, n = odd.neg[c] & b;
                        if (a) o[k] = 0x7f800000u;
                        if (n) o[k] = 0xff800000u;
                        if ((odd.nan[c] & b) || (a && n)) o[k] = 0x7fffffffu;
                    }
                }
                if (store && whole) {
                    uint32_t pk[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        pk[k] = pack_bf16x2(__uint_as_float(o[2 * k]), __uint_as_float(o[2 * k + 1]));
                    uint4 *dst = reinterpret_cast<uint4 *>(p.out + at * D + 32 * c);
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        dst[u] = make_uint4(pk[4 * u], pk[4 * u + 1], pk[4 * u + 2], pk[4 * u + 3]);
                } else if (store) {
                    uint4 *dst = reinterpret_cast<uint4 *>(p.part_o + at * D + 32 * c);
#pragma unroll
                    for (int u = 0; u < 8; ++u)
                        dst[u] = make_uint4(o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]);
                }
            }
            if (valid) {
                if (whole) {
                    const int64_t token = int64_t(t.q0) + row / p.q.group;
                    p.lse[(int64_t(h) * p.q.group + row % p.q.group) * p.q.rows + token] =
                        (m_ref + log2f(l)) * 0.6931471805599453f;
                } else {
                    p.part_ml[at] = make_float2(m_ref, l);
                }
            }
        }
        }
    } else if (warp < 12) {
        warpgroup_regs_dec<kRegsDequant>();
        // ----------------------------------------------- dequantisation ---
        constexpr int kLanes = D / 16, kRows = 256 / kLanes, kU = kKeys / kRows;
        // a lane's sixteen columns and first row. Of D = 128's two 64-column chunks, whose rows
        // lie on the same banks, eight consecutive lanes take half a row each in two rows, so
        // that neither their reads nor their swizzled stores meet a bank twice
        const int x = tid - 128;
        const int col = D == 128 ? (x & 3) | ((((x >> 2) ^ (x >> 3)) & 1) << 2) : x & 3;
        const int r0 = D == 128 ? 2 * (x >> 4) + ((x >> 2) & 1) : x >> 2;
        // its two 16-byte units in a 128-byte row of their chunk
        const int ua = (((col % 4) * 2) ^ (r0 & 7)) << 4, ub = ua ^ 16;
        uint8_t *const chunk = smem + (col / 4) * Lay::kChunkBytes + r0 * 128;
        auto store = [&](uint8_t *dst, const uint4 &w, uint32_t sc, bool values) {
            uint32_t o[8];
            if (!widen16(w, sc, o)) {
                const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const uint2 z = widen4_any(ws[y], sc, values, &sb.odd_values);
                    o[2 * y] = z.x;
                    o[2 * y + 1] = z.y;
                }
            }
            *reinterpret_cast<uint4 *>(dst + ua) = make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4 *>(dst + ub) = make_uint4(o[4], o[5], o[6], o[7]);
        };
        static_assert(kRows % 8 == 0, "a lane's rows swizzle alike");
        for (int32_t i = 0; i < sl.ntiles; ++i) {
            const int st = i % S, rs = i % Lay::kRawStages;
            const uint8_t *raw = smem + Lay::kRaw0 + rs * Lay::kRawBytes;
            if (!mbar_wait(&sb.raw_full[rs], (i / Lay::kRawStages) & 1, abort)) break;
            const uint32_t there = sb.there[i % 16];
            uint4 kw[kU], vw[kU];
            uint32_t ks[kU], vs[kU];
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int r = r0 + kRows * u;
                kw[u] = *reinterpret_cast<const uint4 *>(raw + r * D + col * 16);
                vw[u] = *reinterpret_cast<const uint4 *>(raw + Lay::kRawV + r * D + col * 16);
                ks[u] = raw[Lay::kRawKs + r * (D / 32) + col / 2];
                vs[u] = raw[Lay::kRawVs + r * (D / 32) + col / 2];
            }
            if (there != 0x10101010u) { // zeros where there is no slot
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    const int r = r0 + kRows * u;
                    if ((r & 15) >= int((there >> (8 * (r >> 4))) & 0xffu)) {
                        kw[u] = vw[u] = make_uint4(0u, 0u, 0u, 0u);
                        ks[u] = vs[u] = 127;
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sb.raw_empty[rs]);
            if (!mbar_wait(&sb.empty[st], ((i / S) & 1) ^ 1, abort)) break;
            uint8_t *dst = chunk + 2 * st * Lay::kTileBytes;
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                store(dst + u * kRows * 128, kw[u], ks[u], false);
                store(dst + Lay::kTileBytes + u * kRows * 128, vw[u], vs[u], true);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sb.full[st]);
        }
    } else {
        // warps 12-15 (one warpgroup: copies, MMA, two idle) hand registers to the softmax
        warpgroup_regs_dec<kRegsMma>();
        if (warp == kCopyWarp) {
            // ------------------------------------------------- bulk copies ---
            // lane 4 x + y copies array y (K, V, their scales) of piece x: a page's slots of this
            // head, or the half of a 128-slot page that the tile covers
            const int32_t slots = min(size, kKeys), piece = lane >> 2, array = lane & 3;
            const bool mine = piece < kKeys / slots;
            const uint8_t *const src = array == 0   ? p.c.k
                                       : array == 1 ? p.c.v
                                       : array == 2 ? p.c.k_scales
                                                    : p.c.v_scales;
            const uint32_t row_bytes = array < 2 ? D : D / 32;
            const uint32_t offset =
                (array == 0 ? 0 : array == 1 ? Lay::kRawV : array == 2 ? Lay::kRawKs : Lay::kRawVs) +
                piece * slots * row_bytes;
            auto slot_of = [&](int32_t i) {
                return sl.listed ? unit_slot(sl, sb, i, piece) : sl.from + i * kKeys + piece * slots;
            };
            // (the first tile may begin with pages that no row needs and that may be gone)
            auto wanted = [&](int32_t us) { return mine && us < sl.end && us + slots > sl.first; };
            auto entry_of = [&](int32_t i) -> int32_t { // page table entry, not checked yet
                if (i >= sl.ntiles) return -1;
                const int32_t us = slot_of(i);
                return wanted(us) ? __ldg(p.c.page_table + int64_t(t.b) * p.c.max_pages + (us >> p.c.page_shift)) : -1;
            };
            int32_t next = entry_of(0), i = 0;
            for (; i < sl.ntiles; ++i) {
                const int rs = i % Lay::kRawStages;
                const int32_t id = next;
                next = entry_of(i + 1);
                int32_t count = 0; // slots of the piece that there are
                const int32_t us = slot_of(i);
                if (uint32_t(id) < uint32_t(p.c.num_pages)) count = min(sl.end - us, slots);
                else if (wanted(us)) {
                    cache_range_error(p.c);
                    sb.holes = 1;
                }
                uint32_t there = 0;
                if (mine && array == 0)
                    for (int32_t g = 0; g < slots / 16; ++g)
                        there |= uint32_t(max(0, min(16, count - 16 * g))) << (8 * (piece * (slots / 16) + g));
                there = __reduce_or_sync(0xffffffffu, there);
                __syncwarp(); // (holes, before lane 0 arrives)
                const uint32_t bytes = count > 0 ? slots * row_bytes : 0;
                const uint32_t total = __reduce_add_sync(0xffffffffu, bytes);
                if (!mbar_wait(&sb.raw_empty[rs], ((i / Lay::kRawStages) & 1) ^ 1, abort)) break;
                if (lane == 0) {
                    sb.there[i % 16] = there;
                    mbar_arrive_expect_tx(&sb.raw_full[rs], total);
                }
                __syncwarp();
                if (bytes)
                    bulk_load(smem + Lay::kRaw0 + rs * Lay::kRawBytes + offset,
                              src + cache_row(p.c, id, h, us & (size - 1)) * row_bytes, bytes, &sb.raw_full[rs]);
            }
            // no copy may be under way when the block ends (after a timed-out wait, too)
            int late = 0;
            for (int32_t j = max(0, i - Lay::kRawStages); j < i; ++j)
                mbar_wait(&sb.raw_full[j % Lay::kRawStages], (j / Lay::kRawStages) & 1, &late);
        } else if (warp == kMmaWarp) {
            // ---------------------------------------------------- MMA issue ---
            constexpr uint32_t idesc_s = idesc_bf16(128, kKeys, false, false);
            constexpr uint32_t idesc_o = idesc_bf16(128, D, false, true);
            for (int32_t i = 0; i < sl.ntiles; ++i) {
                const int st = i % S;
                const uint32_t k_addr = smem_base + 2 * st * Lay::kTileBytes, v_addr = k_addr + Lay::kTileBytes;
                if (!mbar_wait(&sb.full[st], (i / S) & 1, abort)) break;
                tc_fence_after();
                // S over the previous tile's P, whose P V was issued before it
    #pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    mma_ts(tmem + Lay::kColS, tmem + Lay::kColQ + kk * 8,
                           sdesc_sw128(k_addr + (kk / 4) * Lay::kChunkBytes + (kk % 4) * 32, 16, 1024), idesc_s,
                           kk > 0 ? 1u : 0u);
                tc_commit(&sb.s_full);
                __syncwarp();
                if (!mbar_wait(&sb.p_full, i & 1, abort)) break;
                tc_fence_after();
    #pragma unroll
                for (int kk = 0; kk < kKeys / 16; ++kk)
                    mma_ts(tmem + Lay::kColO, tmem + Lay::kColS + kk * 8,
                           sdesc_sw128(v_addr + kk * 2048, Lay::kChunkBytes, 1024), idesc_o,
                           (i > 0 || kk > 0) ? 1u : 0u);
                tc_commit(&sb.empty[st]);
                if (i + 1 == sl.ntiles) tc_commit(&sb.o_final);
                __syncwarp();
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, Lay::kTmemCols);
    if (tid == 0 && sb.abort && p.c.status) atomicOr(p.c.status, kStatusTimeout);
}

template <int D>
cudaError_t launch_cache_fwd_mma(const CacheFwd &p, const CacheFwdPlan &plan, cudaStream_t stream)
{
    auto kern = cache_fwd_mma_kernel<D>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, MmaLayout<D>::kAlloc);
    if (e != cudaSuccess) return e;
    // the register split only works if the block is launched with at least the budgets' sum
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, kern);
    if (e != cudaSuccess) return e;
    if (fa.numRegs * kThreads < int(128 * (kRegsSoftmax + 2 * kRegsDequant + kRegsMma)))
        return cudaErrorInvalidConfiguration;
    const dim3 grid(unsigned(plan.tiles), unsigned(p.c.kv_heads), unsigned(p.nsplit));
    kern<<<grid, kThreads, MmaLayout<D>::kAlloc, stream>>>(p);
    return cudaGetLastError();
}

template cudaError_t launch_cache_fwd_mma<64>(const CacheFwd &, const CacheFwdPlan &, cudaStream_t);
template cudaError_t launch_cache_fwd_mma<128>(const CacheFwd &, const CacheFwdPlan &, cudaStream_t);

} // namespace ba
