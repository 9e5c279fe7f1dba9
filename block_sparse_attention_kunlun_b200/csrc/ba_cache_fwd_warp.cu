// Attention over the history cache for a few query rows of a key/value head (2 to 16: one
// event under grouped heads, small trees and candidate sets). The rule, the tiles and the
// splits are ba_cache_fwd.cu's.
//
// With so few rows the bytes of the cache are the bound, and widening their codes is the work:
// it must be done once for all rows of a tile and go no further than registers. A 128-row
// tcgen05 tile would be all but empty, and its operand would have to cross shared memory (387
// us where this kernel's HBM floor is 148: one event under four query heads a key/value head
// over 16 histories of some 28,000); on the CUDA cores each row pays its own products (the
// same 386 us). So each warp takes 16 slots at a time with the warp-wide m16n8k16 MMA, whose
// fragments live in registers:
//   S^T [16 slots x 8 rows] = K Q^T: a lane widens the codes of two slots for the A fragment.
//       The order of a contraction's columns is free, so a lane's four consecutive codes serve
//       as its four columns of a step (Q's fragment is loaded in the same order once);
//   O^T [16 columns x 8 rows] += V^T P^T: a lane reads 16 consecutive codes of four slots and
//       pairs them slot by slot; which of the output's rows stands for which column is free
//       too. P^T comes from S^T by movmatrix.
// Codes are widened to bf16, exactly (as in ba_cache_fwd_sm100.cu); P is rounded to bf16, as in ba_fwd
// (its sum is not): out is then off by 0.0019 to 0.0020 of its size (root mean square) where its own
// rounding to bf16 makes 0.0016. P in two bf16 parts, with twice the MMAs of P V, would end at 0.0016
// and take 5% longer under four heads, 7% under sixteen. Values
// are on their way while S is formed, the next slots' keys while P V is. Slots with codes that the
// widening does not know (NaN, scales past 2^7) get their scores, and their values, put in in
// float32 after the MMAs: everything else stays the same to the bit.
//
// The case above: 0.97 GB in 219 to 229 us, 4.2 to 4.4 TB/s; with sixteen query heads 302 to 313. No unit
// is busy all the time: ncu has the integer pipe at 58%, issue at 59% and DRAM at 54%, with 22% of an SM's
// warps. To put a code's bits into a bf16's places takes four integer operations for two codes, the most of the
// integer pipe's time, with loads and MMAs that wait for one another between them. (NaN looked for in the codes
// ahead of the MMAs: 234 and
// 351; a step's loads all at once: 240 and 411; widened by the float16 conversion instruction:
// 285; with the pages brought into L2 ahead: 267.)
#include "ba_cache_fwd.cuh"
#include "ba_kernels.cuh"
#include "ba_ptx.cuh"

namespace ba {

namespace {

constexpr int kWarpCount = 4;

__device__ __forceinline__ void mma_16x8x16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Four codes c0 .. c3 as the bf16 pairs (c0, c2) and (c1, c3), each times its half of `factor`:
// sign, exponent and mantissa moved to a bf16's places are the value times 2^-120. `top` keeps
// the largest magnitudes so far, in both halves (see_nan).
__device__ __forceinline__ void widen4(uint32_t w, uint32_t factor, uint32_t &even, uint32_t &odd, uint32_t &top)
{
    const uint32_t mx = (w << 4) & 0x07f007f0u, my = (w >> 4) & 0x07f007f0u;
    const uint32_t x = mx | ((w << 8) & 0x80008000u);
    const uint32_t y = my | (w & 0x80008000u);
    top = __vimax3_u16x2(top, mx, my);
    const __nv_bfloat162 f = *reinterpret_cast<const __nv_bfloat162 *>(&factor);
    const __nv_bfloat162 a = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&x), f);
    const __nv_bfloat162 b = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&y), f);
    even = *reinterpret_cast<const uint32_t *>(&a);
    odd = *reinterpret_cast<const uint32_t *>(&b);
}

// 2^(code - 127 + 120) as a bf16 (codes up to 134).
__device__ __forceinline__ uint32_t bf16_factor(uint32_t code) { return (code << 7) + 0x3c00u; }

// Whether a code widened into `top` was NaN (0x7f0; it was taken for 480).
__device__ __forceinline__ bool see_nan(uint32_t top) { return ((top + 0x08100810u) & 0x10001000u) != 0; }

// A byte of `nan_bits` has its top bit set when the code there is NaN.
__device__ __forceinline__ uint32_t nan_bits(uint32_t w) { return (w & 0x7f7f7f7fu) + 0x01010101u; }

// 16 slots' codes and scale codes as one lane (g = lane / 4, t = lane % 4) holds them.
template <int D>
struct KeyCodes {
    static constexpr int kWords = D / 16;
    uint32_t w[2][kWords]; // slots g, g + 8: 16 codes from 16 t on (D = 128: and from 64 + 16 t on)
    uint32_t scales[2];    // the slots' scale codes, a byte a block

    // codes, scale codes: this lane's first ones of slot 0, `row` slots before these
    __device__ __forceinline__ void load(const uint8_t *codes, const uint8_t *scale_codes, int64_t row)
    {
        const uint8_t *const c = codes + row * D, *const s = scale_codes + row * (D / 32);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int x = 0; x < D / 64; ++x) {
                const uint4 v = __ldg(reinterpret_cast<const uint4 *>(c + 8 * i * D + 64 * x));
                w[i][4 * x] = v.x, w[i][4 * x + 1] = v.y, w[i][4 * x + 2] = v.z, w[i][4 * x + 3] = v.w;
            }
            if constexpr (D == 128) scales[i] = __ldg(reinterpret_cast<const uint32_t *>(s + 8 * i * (D / 32)));
            else scales[i] = __ldg(reinterpret_cast<const uint16_t *>(s + 8 * i * (D / 32)));
        }
    }
};

template <int D>
struct ValueCodes {
    static constexpr int kWords = D / 32;
    uint32_t w[4][kWords]; // slots 2 t, 2 t + 1, 2 t + 8, 2 t + 9: D / 8 codes from D / 8 g on
    uint32_t scale[4];     // scale codes of the codes' block

    __device__ __forceinline__ void load(const uint8_t *codes, const uint8_t *scale_codes, int64_t row)
    {
        const uint8_t *const c = codes + row * D, *const s = scale_codes + row * (D / 32);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = (i & 1) + 8 * (i >> 1);
            if constexpr (D == 128) {
                const uint4 v = __ldg(reinterpret_cast<const uint4 *>(c + at * D));
                w[i][0] = v.x, w[i][1] = v.y, w[i][2] = v.z, w[i][3] = v.w;
            } else {
                const uint2 v = __ldg(reinterpret_cast<const uint2 *>(c + at * D));
                w[i][0] = v.x, w[i][1] = v.y;
            }
            scale[i] = __ldg(s + at * (D / 32));
        }
    }
};

// One lane's share of a tile's softmax: rows 2 t and 2 t + 1 of each eight. o[n][j]: columns
// d = D / 8 g + 2 j (first two values) and d + 1 (last two) of rows 8 n + 2 t and 8 n + 2 t + 1.
template <int D, int kN>
struct Share {
    float m[kN / 8][2], l[kN / 8][2]; // m: the rows' maximum (log2), the same in all lanes of a row; l: this lane's slots
    float o[kN / 8][D / 16][4];
};

// q . k in float32 from memory, for a slot with codes that widen4 does not know.
template <int D>
__device__ __noinline__ float score_any(const __nv_bfloat16 *q, const uint8_t *k, const uint8_t *scales)
{
    float sum = 0.f;
    for (int d = 0; d < D; ++d)
        sum = fmaf(__bfloat162float(q[d]), e4m3x2_to_f32(__ldg(k + d)).x * mx_scale(__ldg(scales + d / 32)), sum);
    return sum;
}

} // namespace

template <int D, int kN>
__global__ void __launch_bounds__(kWarpCount * 32, kN == 8 ? 4 : 3)
    cache_fwd_warp_kernel(const __grid_constant__ CacheFwd p)
{
    constexpr int kTiles = kN / 8;
    __shared__ float sm_o[kWarpCount][kN][D + 4];
    __shared__ float2 sm_ml[kWarpCount][kN];
    __shared__ RowView views[kN];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t4 = lane & 3;
    const int32_t h = blockIdx.y, split = blockIdx.z;
    FwdTile t;
    if (!find_tile(p, blockIdx.x, kN, t)) return;

    // the rows' views, and Q's fragments: row g of each eight, in the codes' order
    if (threadIdx.x < kN) views[threadIdx.x] = row_view(p, t, t.row0 + min(int(threadIdx.x), t.rows - 1));
    __syncthreads();
    uint32_t q[kTiles][D / 16][2];
    int32_t min_ws, max_ws, min_pos, max_pos;
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
        const uint4 *src = reinterpret_cast<const uint4 *>(
            p.q.q + out_row(p, t, h, t.row0 + min(8 * n + g, t.rows - 1)) * D + 16 * t4);
#pragma unroll
        for (int x = 0; x < D / 64; ++x)
#pragma unroll
            for (int u = 0; u < 2; ++u) { // eight columns: two of the lane's words of codes
                const uint4 w = __ldg(src + 8 * x + u);
                q[n][4 * x + 2 * u][0] = __byte_perm(w.x, w.y, 0x5410);
                q[n][4 * x + 2 * u][1] = __byte_perm(w.x, w.y, 0x7632);
                q[n][4 * x + 2 * u + 1][0] = __byte_perm(w.z, w.w, 0x5410);
                q[n][4 * x + 2 * u + 1][1] = __byte_perm(w.z, w.w, 0x7632);
            }
    }
    {
        const RowView v = views[lane % kN];
        min_ws = __reduce_min_sync(0xffffffffu, v.ws);
        max_ws = __reduce_max_sync(0xffffffffu, v.ws);
        min_pos = __reduce_min_sync(0xffffffffu, v.pos);
        max_pos = __reduce_max_sync(0xffffffffu, v.pos);
    }

    // this split's slots, in groups of 16
    const int32_t lo = first_slot(p, t, min_ws) / kGroup * kGroup;
    int64_t from = lo + int64_t(split) * p.chunk, to = split + 1 == p.nsplit ? t.end : from + p.chunk;
    if (to > t.end) to = t.end;
    // `from` is a multiple of 16; a split that starts past the end has nothing
    const int32_t g1 = int32_t((to + kGroup - 1) / kGroup), g0 = from < t.end ? int32_t(from / kGroup) : g1;

    Share<D, kN> s;
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
#pragma unroll
        for (int r = 0; r < 2; ++r) s.m[n][r] = -INFINITY, s.l[n][r] = 0.f;
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) s.o[n][j][e] = 0.f;
    }

    // walk of this warp's groups: 32 at a time are tested for being wanted by any row
    const int32_t tok0 = t.row0 / p.q.group, tok1 = (t.row0 + t.rows - 1) / p.q.group;
    int32_t base = g0 - kWarpCount * 32, id = -1;
    uint32_t todo = 0;
    auto next_group = [&](int32_t &slot, int64_t &row) -> bool {
        while (!todo) {
            base += kWarpCount * 32;
            if (base >= g1) return false;
            const int32_t gr = base + lane * kWarpCount + warp, s0 = gr * kGroup;
            bool want = gr < g1 && (s0 + kGroup > min_ws || s0 + kGroup > t.len);
            if (gr < g1 && !want && p.page_mask) {
                const int32_t page = s0 >> p.c.page_shift;
                for (int32_t tok = tok0; tok <= tok1 && !want; ++tok)
                    want = (__ldg(p.page_mask + ((int64_t(t.q0) + tok) * p.c.kv_heads + h) * p.mask_words +
                                  (page >> 5)) >>
                            (page & 31)) & 1u;
            }
            want = want && (s0 <= max_pos || s0 + kGroup > t.len);
            id = -1;
            if (want) {
                id = cache_page(p.c, t.b, s0 >> p.c.page_shift);
                if (id < 0) cache_range_error(p.c);
            }
            todo = __ballot_sync(0xffffffffu, id >= 0);
        }
        const int x = __ffs(todo) - 1;
        todo &= todo - 1;
        slot = (base + x * kWarpCount + warp) * kGroup;
        row = int64_t(__shfl_sync(0xffffffffu, id, x)) * (p.c.kv_heads << p.c.page_shift) +
              ((h << p.c.page_shift) + (slot & ((1 << p.c.page_shift) - 1)));
        return true;
    };

    const uint8_t *const k_codes = p.c.k + g * D + 16 * t4, *const k_scales = p.c.k_scales + g * (D / 32);
    const uint8_t *const v_codes = p.c.v + 2 * t4 * D + D / 8 * g;
    const uint8_t *const v_scales = p.c.v_scales + 2 * t4 * (D / 32) + g / (256 / D);
    const int32_t inside = min(min_pos, t.len - 1) - (kGroup - 1); // last slot whose 16 all rows see
    KeyCodes<D> keys;
    ValueCodes<D> values;
    int32_t next_slot;
    int64_t next_row;
    bool more = next_group(next_slot, next_row);
    if (more) keys.load(k_codes, k_scales, next_row);
    while (more) {
        const int32_t slot = next_slot;
        const int64_t row = next_row;
        values.load(v_codes, v_scales, row);
        const bool all = slot >= max_ws && slot <= inside;
        // S^T
        float sc[kTiles][4];
#pragma unroll
        for (int n = 0; n < kTiles; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.f;
        uint32_t top[2] = {0, 0};
#pragma unroll
        for (int x = 0; x < KeyCodes<D>::kWords; ++x) {
            // block of the word's columns: (16 t + 64 (x / 4)) / 32
            const int shift = 8 * (t4 / 2 + 2 * (x / 4));
            uint32_t a[4];
            widen4(keys.w[0][x], bf16_factor((keys.scales[0] >> shift) & 0xffu) * 0x00010001u, a[0], a[2], top[0]);
            widen4(keys.w[1][x], bf16_factor((keys.scales[1] >> shift) & 0xffu) * 0x00010001u, a[1], a[3], top[1]);
#pragma unroll
            for (int n = 0; n < kTiles; ++n) mma_16x8x16(sc[n], a, q[n][x][0], q[n][x][1]);
        }
        // Slots with codes that the widening does not know: their scores, which no other slot's depend
        // on, are formed again below. (A scale code over 134: its byte plus 121 carries into bit 8 of
        // a 16-bit field.)
        uint32_t odd_keys = 0;
        {
            bool odd[2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                odd[i] = see_nan(top[i]) || ((((keys.scales[i] & 0x00ff00ffu) + 0x00790079u) |
                                              (((keys.scales[i] >> 8) & 0x00ff00ffu) + 0x00790079u)) & 0x01000100u);
            if (__any_sync(0xffffffffu, odd[0] || odd[1]))
                odd_keys = __reduce_or_sync(0xffffffffu, uint32_t(odd[0]) << g | uint32_t(odd[1]) << (g + 8));
        }
        // softmax: values 0, 1 are slot g's for rows 2 t, 2 t + 1, values 2, 3 slot g + 8's
        more = next_group(next_slot, next_row);
        if (more) keys.load(k_codes, k_scales, next_row);
        if (odd_keys) {
#pragma unroll 1
            for (int i = 0; i < 2; ++i) {
                if (!((odd_keys >> (g + 8 * i)) & 1u)) continue;
                const int64_t r8 = row + g + 8 * i;
#pragma unroll
                for (int n = 0; n < kTiles; ++n)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int32_t at = t.row0 + min(8 * n + 2 * t4 + r, t.rows - 1);
                        const float x = score_any<D>(p.q.q + out_row(p, t, h, at) * D, p.c.k + r8 * D,
                                                     p.c.k_scales + r8 * (D / 32));
                        if (i == 0) sc[n][r] = x;
                        else sc[n][2 + r] = x;
                    }
            }
            __syncwarp();
        }
        uint32_t b[kTiles][2];
        bool grow = false;
#pragma unroll
        for (int n = 0; n < kTiles; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                sc[n][e] *= p.scale_log2;
                if (!all) {
                    const int32_t k = slot + g + 8 * (e >> 1);
                    if (!(k < t.end && sees(p, t, views[8 * n + 2 * t4 + (e & 1)], h, k))) sc[n][e] = -INFINITY;
                }
                grow |= sc[n][e] > s.m[n][e & 1] + 8.f;
            }
        // O and l move to a new maximum only when a score exceeds the old one by more than 8
        // (P stays below 2^8)
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int n = 0; n < kTiles; ++n)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float top = fmaxf(sc[n][r], sc[n][2 + r]);
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                    // (each row by itself: another row's scores must not change its roundings)
                    const float m = top > s.m[n][r] + 8.f ? top : s.m[n][r];
                    const float alpha = ex2_approx(s.m[n][r] - (m == -INFINITY ? 0.f : m));
                    s.m[n][r] = m;
                    s.l[n][r] *= alpha;
#pragma unroll
                    for (int j = 0; j < D / 16; ++j) {
                        s.o[n][j][r] *= alpha;
                        s.o[n][j][2 + r] *= alpha;
                    }
                }
        }
#pragma unroll
        for (int n = 0; n < kTiles; ++n) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float m = s.m[n][e & 1];
                sc[n][e] = ex2_approx(sc[n][e] - (m == -INFINITY ? 0.f : m));
                s.l[n][e & 1] += sc[n][e];
            }
            b[n][0] = transpose_8x8(pack_bf16x2(sc[n][0], sc[n][1]));
            b[n][1] = transpose_8x8(pack_bf16x2(sc[n][2], sc[n][3]));
        }
        // Values under scales that the widening does not know take part as zeros. (NaN codes do as 480,
        // which a row that does not see them multiplies by 0.)
        uint32_t odd_values = 0;
        {
            uint32_t high = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) high |= values.scale[i] + 0x79u;
            if (__any_sync(0xffffffffu, high & 0x100u)) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (values.scale[i] > 134) {
#pragma unroll
                        for (int x = 0; x < ValueCodes<D>::kWords; ++x) values.w[i][x] = 0;
                        values.scale[i] = 0;
                        odd_values |= 1u << (2 * t4 + (i & 1) + 8 * (i >> 1));
                    }
                odd_values = __reduce_or_sync(0xffffffffu, odd_values);
            }
        }
        // O^T: slots 2 t, 2 t + 1 in the low and high halves of one register, 2 t + 8 and 2 t + 9 of
        // the other
        const uint32_t f0 = bf16_factor(values.scale[0]) | bf16_factor(values.scale[1]) << 16;
        const uint32_t f1 = bf16_factor(values.scale[2]) | bf16_factor(values.scale[3]) << 16;
        top[0] = 0;
#pragma unroll
        for (int x = 0; x < ValueCodes<D>::kWords; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y) { // columns 4 x + 2 y, 4 x + 2 y + 1 of the lane's
                uint32_t a[4];
                widen4(__byte_perm(values.w[0][x], values.w[1][x], y ? 0x7632 : 0x5410), f0, a[0], a[1], top[0]);
                widen4(__byte_perm(values.w[2][x], values.w[3][x], y ? 0x7632 : 0x5410), f1, a[2], a[3], top[0]);
#pragma unroll
                for (int n = 0; n < kTiles; ++n) mma_16x8x16(s.o[n][2 * x + y], a, b[n][0], b[n][1]);
            }
        if (__any_sync(0xffffffffu, see_nan(top[0]))) {
            uint32_t slots = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t nan = 0;
#pragma unroll
                for (int x = 0; x < ValueCodes<D>::kWords; ++x) nan |= nan_bits(values.w[i][x]);
                if (nan & 0x80808080u) slots |= 1u << (2 * t4 + (i & 1) + 8 * (i >> 1));
            }
            odd_values |= __reduce_or_sync(0xffffffffu, slots);
        }
        // the values that the MMAs did not know, for the rows that see them
        while (odd_values) {
            const int k = __ffs(odd_values) - 1;
            odd_values &= odd_values - 1;
#pragma unroll
            for (int n = 0; n < kTiles; ++n)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float w = __shfl_sync(0xffffffffu, k < 8 ? sc[n][r] : sc[n][2 + r], 4 * (k & 7) + t4);
                    if (slot + k >= t.end || !sees(p, t, views[8 * n + 2 * t4 + r], h, slot + k)) continue;
#pragma unroll
                    for (int j = 0; j < D / 16; ++j)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int d = D / 8 * g + 2 * j + e;
                            const uint32_t code = __ldg(p.c.v + (row + k) * D + d);
                            const uint32_t scale = __ldg(p.c.v_scales + (row + k) * (D / 32) + d / 32);
                            if ((code & 0x7fu) == 0x7fu || scale > 134)
                                s.o[n][j][2 * e + r] =
                                    fmaf(w, e4m3x2_to_f32(code).x * mx_scale(scale), s.o[n][j][2 * e + r]);
                        }
                }
            __syncwarp();
        }
    }

    // the lanes of a row (which share m) join their sums, then the warps everything
#pragma unroll
    for (int n = 0; n < kTiles; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = 8 * n + 2 * t4 + r;
            float l = s.l[n][r];
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
            if (g == 0) sm_ml[warp][row] = make_float2(s.m[n][r], l);
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
                *reinterpret_cast<float2 *>(&sm_o[warp][row][D / 8 * g + 2 * j]) =
                    make_float2(s.o[n][j][r], s.o[n][j][2 + r]);
        }
    __syncthreads();
    const int64_t heads = int64_t(p.c.kv_heads) * p.q.group;
    for (int x = threadIdx.x; x < t.rows * (D / 4); x += kWarpCount * 32) {
        const int r = x / (D / 4), d = x % (D / 4) * 4;
        float mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarpCount; ++w) mx = fmaxf(mx, sm_ml[w][r].x);
        const float ref = mx == -INFINITY ? 0.f : mx;
        float sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarpCount; ++w) {
            const float a = ex2_approx(sm_ml[w][r].x - ref);
            if (sm_ml[w][r].y == 0.f) continue; // saw nothing
            sum = fmaf(sm_ml[w][r].y, a, sum);
            const float4 o = *reinterpret_cast<const float4 *>(&sm_o[w][r][d]);
            acc.x = fmaf(o.x, a, acc.x);
            acc.y = fmaf(o.y, a, acc.y);
            acc.z = fmaf(o.z, a, acc.z);
            acc.w = fmaf(o.w, a, acc.w);
        }
        const int32_t row = t.row0 + r;
        const int64_t oh = out_row(p, t, h, row);
        if (p.nsplit == 1) {
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            *reinterpret_cast<uint2 *>(p.out + oh * D + d) =
                make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
            if (d == 0)
                p.lse[(int64_t(h) * p.q.group + row % p.q.group) * p.q.rows + t.q0 + row / p.q.group] =
                    (mx + log2f(sum)) * 0.6931471805599453f;
        } else {
            const int64_t at = int64_t(split) * p.q.rows * heads + oh;
            *reinterpret_cast<float4 *>(p.part_o + at * D + d) = acc;
            if (d == 0) p.part_ml[at] = make_float2(mx, sum);
        }
    }
}

template <int D>
cudaError_t launch_cache_fwd_warp(const CacheFwd &p, const CacheFwdPlan &plan, cudaStream_t stream)
{
    const dim3 grid(unsigned(plan.tiles), unsigned(p.c.kv_heads), unsigned(p.nsplit));
    if (plan.tile_rows == 8) cache_fwd_warp_kernel<D, 8><<<grid, kWarpCount * 32, 0, stream>>>(p);
    else cache_fwd_warp_kernel<D, 16><<<grid, kWarpCount * 32, 0, stream>>>(p);
    return cudaGetLastError();
}

template cudaError_t launch_cache_fwd_warp<64>(const CacheFwd &, const CacheFwdPlan &, cudaStream_t);
template cudaError_t launch_cache_fwd_warp<128>(const CacheFwd &, const CacheFwdPlan &, cudaStream_t);

} // namespace ba
