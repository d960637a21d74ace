// kv_attention.cuh -- attention over the paged 8-bit cache for few query rows
// per cache head (decode, drafted tokens), and for any number of them with heads of
// more than 128 values: one pass over the cache on mma.sync, work cut along the
// tokens and joined.
//
//   y = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q.k_j),  k_j = sk code, v_j = sv code,
// with one scale sk, sv per page and head.  A row's scores in powers of two,
//   x_j = (scale log2 e) sk (q.code_j) + log2 sv,  m = max x_j,  p'_j = 2^(x_j - m),
// carry the scale of the values: the second product then takes codes, y =
// sum p' code / sum (p' / sv), and p' <= 1 whatever the scales are.  Where a page's
// scale is far below another's, p' may vanish although p does not (a page of zeros
// has 2^-100): the sum then has a reference of its own, see far_scale.
//
// What bounds it: the reading of the codes (2 dim bytes per token and head).
// They enter the tensor cores as exact fp16 values (one conversion per two
// codes), the queries as fp16 times a power of two per row, fp32 queries as
// the sum of two fp16 values.  The tokens are the M side of both products, so
// that eight query rows fill an instruction:
//   S^T [16 tokens x 8 rows]  = K [16 x dim] q^T,
//   O^T [16 dims x 8 rows]   += V^T [16 x 128 tokens] P^T.
// Eight warps share a tile of 128 tokens: each takes 16 tokens of S, and after
// the probabilities went through shared memory 16 (or 32) dims of O, so nobody
// has to add up accumulators but across cut units.  A ninth warp brings the tiles
// by TMA, page by page, in the swizzle that the loads of the fragments want, and
// runs ahead across units.
//
// Measured (8 heads of 128 in the cache, 32 of the queries): 64 sequences of 4096 tokens, one
// row each, 94 us, 5.7 TB/s of codes; one of 32768 22 us, of which the tiles take 6, the
// rest start (shares, page table, queries, first tile: 3) and join (5).  A tile takes 2000
// cycles, two blocks on a multiprocessor beside each other.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "kv_device.cuh"
#include "qmm_internal.h"

namespace qk {

namespace kv {

constexpr int TILE = 128;     // tokens of a tile
constexpr int THREADS = 256;  // 8 warps, and one for the copies
constexpr int LEAST = 2;      // tiles per block below which fewer blocks take part
constexpr int SCALES = 24;    // floats of a tile's scales: of 8 groups of tokens those of keys, log2 and inverse of those of
                              // values (0: see far_scale)
constexpr int SHORT = 4;      // tiles of a unit that is not cut: it goes to the block where it begins

// A power of two on p', so that its low part in fp16 keeps 2^-38 of the largest.
constexpr float P_SHIFT = 14.0f;
// and one on the sum of p' / sv, which then stays within fp32 for 2^31 tokens
// of any scale from 2^-100 to 2^120
constexpr float L_FACTOR = 0x1p-20f;
constexpr float LN2 = 0.6931471805599453f;

struct AttnParams {
    const uint8_t *codes[2];
    const float *scales[2];
    int64_t pages;
    int heads, page, dim, group;  // group: query heads per cache head
    const void *q;
    int64_t ldq_t, ldq_h;
    int q_type, y_type;
    void *y;
    int64_t ldy_t, ldy_h;
    const int32_t *offsets, *lengths, *table;
    int64_t ld_table, T;
    int width, B;
    float factor, factor_low;  // scale * log2 e, and what that loses in 32 bits
    int causal, window;
    uint32_t div_mul, div_shift;  // row / group = row * div_mul >> div_shift for rows below 2^31
    float *lse;
    float *part;
    unsigned *count;
    int *status;
    int stop;  // the tile at which the first CTA's copies stop (NO_STOP: none)
};

// A sequence of the batch and its share of the work: `units` = heads x row
// blocks, each of `tiles` tiles from token lo (a multiple of TILE) on.
struct Seq {
    int row0, n, len, lo, tiles, blocks;
    int64_t units;
};

// a / b of what is mostly below 2^32 (a 64-bit division takes hundreds of cycles).
__device__ __forceinline__ long long divide(long long a, long long b) {
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}
// The row of the batch (within its sequence) of query row r < 2^31.
__device__ __forceinline__ int token_of(const AttnParams &P, int r) {
    return static_cast<int>(static_cast<uint64_t>(r) * P.div_mul >> P.div_shift);
}

// The first token that the row at position pos of its sequence sees (pos - window + 1
// may lie below -2^31: rows before the first token, windows near 2^31).
__device__ __forceinline__ int seen_from(const AttnParams &P, int pos) {
    return P.window ? max(pos, P.window - 1) - (P.window - 1) : 0;
}

template <int R>
__device__ __forceinline__ bool load_seq(const AttnParams &P, int b, Seq &s) {
    s.units = 0;
    s.tiles = 0;
    int lo = b, hi = b + 1;
    if (P.offsets) lo = __ldg(P.offsets + b), hi = __ldg(P.offsets + b + 1);
    const int len = __ldg(P.lengths + b);
    if (lo < 0 || hi < lo || hi > P.T || len < 0 || len > static_cast<int64_t>(P.width) * P.page) return false;
    s.row0 = lo;
    s.n = hi - lo;
    s.len = len;
    if (s.n == 0) return true;
    s.lo = seen_from(P, len - s.n) & ~(TILE - 1);
    s.tiles = max(1, (len - s.lo + TILE - 1) / TILE);
    s.blocks = (s.n * P.group + R - 1) / R;  // (the call's rows times group are below 2^31 - R)
    s.units = static_cast<int64_t>(s.blocks) * P.heads;
    return true;
}

// A box of one page and head: up to 128 bytes of `page` rows from column c on (zeros
// behind dim).
__device__ __forceinline__ void tma_page(uint32_t dst, const CUtensorMap *map, int c, int tile, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c), "r"(0), "r"(tile), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
// Whether one of 16 codes is a NaN.
__device__ __forceinline__ bool has_nan(const uint4 &v) {
    auto nan = [](uint32_t w) { return (w & 0x7f7f7f7fu) + 0x01010101u; };  // bit 7 of a byte is set if it was 0x7f
    return ((nan(v.x) | nan(v.y) | nan(v.z) | nan(v.w)) & 0x80808080u) != 0;
}
// 16 codes with 0 where one is a NaN.
__device__ __forceinline__ uint4 without_nan(const uint4 &v) {
    auto clean = [](uint32_t w) { return w & ~__vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu); };
    return make_uint4(clean(v.x), clean(v.y), clean(v.z), clean(v.w));
}
// The results that NaNs among the values reach, of rows ra .. rb - 1 of the unit (from query
// row r0 on) and dims d0 .. d1 - 1: set(row, dim) for each.  In tiles that some rows see and
// some do not 0 times a NaN would reach all of them, so the kernels take a NaN there for 0, note
// that there was one, and come here once their results are written: the values of tokens from .. to - 1
// are read again, but for those of tiles that all rows see.  By `count` threads, 16 or more.
template <class Set>
__device__ __forceinline__ void spread_nans(const AttnParams &P, int b, int head, int start, int r0, int ra, int rb, int d0, int d1,
                                            int from, int to, int all_lo, int all_hi, int idx, int count, const Set &set) {
    const int chunks = (min(d1, P.dim) - d0) / 16;
    if (chunks <= 0 || ra >= rb) return;
    const int step = count / chunks, chunk = idx % chunks;
    if (idx >= step * chunks) return;
#pragma unroll 1
    for (int64_t k = from + idx / chunks; k < to; k += step) {
        if (k - all_lo >= TILE && all_hi - k > TILE + step) {
            k += (all_hi - TILE - k) / step * step - step;
            continue;
        }
        const int32_t id = __ldg(P.table + static_cast<int64_t>(b) * P.ld_table + k / P.page);
        if (id < 0 || id >= P.pages) continue;
        const int64_t row = (static_cast<int64_t>(id) * P.heads + head) * P.page + k % P.page;
        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(P.codes[1] + row * P.dim + d0) + chunk);
        if (!has_nan(v)) continue;
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll 1
        for (int r = ra; r < rb; ++r) {
            const int pos = start + token_of(P, r0 + r);
            if (k < seen_from(P, pos) || (P.causal && k > pos)) continue;
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if ((w[e / 4] >> (8 * (e & 3)) & 0x7f) == 0x7f) set(r, d0 + 16 * chunk + e);
        }
    }
}
constexpr uint32_t A_NAN = 0x7fffffffu;

// Two codes as exact fp16 values.
__device__ __forceinline__ uint32_t halves(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
    return r;
}
__device__ __forceinline__ uint32_t halves_hi(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(w));
    return r;
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Whether a value scale lies outside 2^-61 .. 2^29.  Within, scales are at most 2^90
// apart, and p' of a score up to 2^35 below the row's largest stays above 2^-126,
// which ex2 would make 0: what is lost of a row's sum is below 2^-35 of its largest
// part for each token.  From the first tile of a unit with such a scale on (its inverse
// scales are 0), the sum is kept apart as a FarSum.
__device__ __forceinline__ bool far_scale(float v) { return !(v >= 0x1p-61f && v <= 0x1p29f); }
// The sum of p without the scales, relative to 2^m of the scores alone.  In memory, as the
// registers are those of the ordinary case.
struct FarSum {
    volatile float m, l;
    // s(i): the score i of n, -inf where it is masked; unit: what p = 1 counts
    template <class S>
    __device__ __forceinline__ void add(int n, float unit, const S &s) {
        const float was = m;
        float top = was;
#pragma unroll
        for (int i = 0; i < n; ++i) top = fmaxf(top, s(i));
        const float ref = top == -INFINITY ? 0.0f : top;  // (nothing was seen yet: any finite one)
        float sum = l * ex2(was - ref);
#pragma unroll
        for (int i = 0; i < n; ++i) sum = fmaf(ex2(s(i) - ref), unit, sum);
        m = top, l = sum;
        asm volatile("" ::: "memory");  // (one after another: side by side they would take more registers)
    }
    // relative to 2^ref, the reference of the row's products
    __device__ __forceinline__ float at(float ref) const { return l != 0.0f ? l * ex2(0.5f * (m - ref)) * ex2(0.5f * (m - ref)) : 0.0f; }
};
// v 2^d for d <= 0, also where 2^d is below fp32 (a sum over scales of 2^-100 is
// large enough to be seen beside one over scales of 2^100).
__device__ __forceinline__ float faded(float v, float d) { return v * ex2(fmaxf(d, -126.0f)) * ex2(fminf(d + 126.0f, 0.0f)); }

__device__ __forceinline__ void store_typed(void *p, int64_t i, int type, float v) {
    if (type == QMM_F32) static_cast<float *>(p)[i] = v;
    else if (type == QMM_F16) static_cast<__half *>(p)[i] = __float2half_rn(v);
    else static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
}

// A query value as it lies in memory, and as fp32.  (A load with its conversion inside a
// branch by type waits for its value: 16 of them one after another took 7300 cycles.)
template <bool F32>
using QueryRaw = typename std::conditional<F32, float, uint16_t>::type;
__device__ __forceinline__ float query_value(float v, int) { return v; }
__device__ __forceinline__ float query_value(uint16_t v, int type) {
    return type == QMM_F16 ? __half2float(__ushort_as_half(v)) : __uint_as_float(static_cast<uint32_t>(v) << 16);
}

// DP: dim rounded up to 64, 128 or 256; NB: groups of eight query rows of a
// block; HL: queries and probabilities as two fp16 parts.
template <int DP, int NB, bool HL>
struct Few {
    static constexpr int R = 8 * NB, PARTS = HL ? 2 : 1, CONSUMERS = THREADS;
    static constexpr float SHIFT = P_SHIFT;
    static constexpr int CTAS = DP == 256 ? 1 : 2;  // per multiprocessor
    static constexpr int STAGES = DP == 64 ? 4 : DP == 128 && NB * PARTS <= 2 ? 3 : 2;  // (two CTAs per multiprocessor up to 128)
    static constexpr int ROW = DP == 64 ? 64 : 128, COLS = DP / ROW;  // bytes of a row of a box, boxes side by side
    static constexpr int SIDE = TILE * DP, STAGE = 2 * SIDE;
    static constexpr int QP = DP + 16, PP = TILE + 16;  // pitches in halves: 8 banks between rows, as 8-byte reads want
    static constexpr int OFF_Q = STAGES * STAGE;
    static constexpr int OFF_P = OFF_Q + PARTS * R * QP * 2;
    static constexpr int OFF_RED = OFF_P + PARTS * R * PP * 2;       // [8 warps][R]
    static constexpr int OFF_ROW = OFF_RED + 8 * R * 4;              // [R] factor of the row, [R] first, [R] end, [R] the factor's low part
    static constexpr int OFF_SC = OFF_ROW + 4 * R * 4;               // [STAGES][SCALES]
    static constexpr int OFF_BAR = (OFF_SC + STAGES * SCALES * 4 + 7) / 8 * 8;
    static constexpr int SMEM = OFF_BAR + 16 * STAGES + 16;  // (barriers, the parts that were there, whether there was a NaN)
    static_assert(CTAS == 1 ? SMEM <= 232448 : 2 * (SMEM + 1024) <= 233472, "shared memory");
    static constexpr int PART = R * (DP + 2);  // floats of a partial result
    // byte of 16-byte chunk c of a row of a tile
    static __device__ __forceinline__ int at(int row, int c) {
        if constexpr (DP == 64) return row * 64 + ((c ^ (row >> 1 & 3)) << 4);
        else return (c >> 3) * (TILE * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4);
    }
};

// Where a CTA's share of the tiles lies: sequence, unit of it, tile of that.
struct Walk {
    int b, tile;
    int64_t unit;
    long long seq0, t;  // tiles before the sequence, and before this one
    Seq s;
};
// On to the next unit, nt tiles further.
template <int R>
__device__ __forceinline__ void advance(const AttnParams &P, Walk &w, int nt, long long t1) {
    w.t += nt;
    w.tile = 0;
    if (w.t < t1 && ++w.unit == w.s.units) {
        w.seq0 += w.s.units * w.s.tiles;
        w.unit = 0;
        do load_seq<R>(P, ++w.b, w.s);
        while (w.s.units == 0);
    }
}
// The rows of a unit, and the tokens and tiles that some of them see.
struct Span {
    int head, nt, r0, rows, lo, hi, all_lo, all_hi;
    int from, jb, je;  // tiles jb .. je - 1 from token `from` on
};
template <int R>
__device__ __forceinline__ Span span_of(const AttnParams &P, const Walk &w, long long t1) {
    Span u;
    const Seq &s = w.s;
    u.head = static_cast<int>(s.blocks == 1 ? w.unit : divide(w.unit, s.blocks));
    const int block = static_cast<int>(w.unit - static_cast<int64_t>(u.head) * s.blocks);
    u.nt = s.tiles <= SHORT ? s.tiles : static_cast<int>(min(static_cast<long long>(s.tiles - w.tile), t1 - w.t));
    u.r0 = block * R;
    u.rows = min(R, s.n * P.group - u.r0);
    const int start = s.len - s.n;
    const int i0 = token_of(P, u.r0), i1 = token_of(P, u.r0 + u.rows - 1);
    u.hi = P.causal ? min(s.len, start + i1 + 1) : s.len;
    u.all_hi = P.causal ? min(s.len, start + i0 + 1) : s.len;
    u.lo = seen_from(P, start + i0);
    u.all_lo = seen_from(P, start + i1);
    u.from = s.lo;
    u.jb = max(w.tile, (u.lo - s.lo) / TILE);
    u.je = min(w.tile + u.nt, u.hi > s.lo ? (u.hi - s.lo + TILE - 1) / TILE : 0);
    return u;
}

// Where this CTA's share of the tiles begins (w.t) and ends (t1), of W tiles in `blocks`
// shares; false: it has none.  Every warp finds it by itself: nobody waits for a
// barrier in the first microseconds, which a small call is made of.
template <int R>
__device__ __forceinline__ bool begin_walk(const AttnParams &P, int lane, Walk &w, long long &t1, long long &W, int &blocks) {
    const int share = (P.B + 31) / 32;
    long long sum = 0;
    for (int b = lane * share; b < min(P.B, (lane + 1) * share); ++b) {
        Seq s;
        if (!load_seq<R>(P, b, s)) atomicOr(P.status, STATUS_INDEX);
        sum += s.units * s.tiles;
    }
    long long before = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += v;
    }
    W = __shfl_sync(0xffffffffu, before, 31);
    before -= sum;
    if (W == 0) return false;
    blocks = static_cast<int>(min(static_cast<long long>(gridDim.x), max(1ll, W / LEAST)));
    const int cta = blockIdx.x;
    if (cta >= blocks) return false;
    t1 = divide((cta + 1) * W, blocks);
    w.t = divide(cta * W, blocks);
    const int from = __ffs(__ballot_sync(0xffffffffu, before <= w.t && w.t < before + sum)) - 1;
    w.b = from * share;
    w.seq0 = __shfl_sync(0xffffffffu, before, from);
    for (;; ++w.b) {
        load_seq<R>(P, w.b, w.s);
        if (w.t < w.seq0 + w.s.units * w.s.tiles) break;
        w.seq0 += w.s.units * w.s.tiles;
    }
    w.unit = divide(w.t - w.seq0, w.s.tiles);
    w.tile = static_cast<int>((w.t - w.seq0) - w.unit * w.s.tiles);
    if (w.tile && w.s.tiles <= SHORT) advance<R>(P, w, w.s.tiles - w.tile, t1);
    return true;
}

// The copies of a CTA's tiles, by one warp.  W: the walk over its units, span_of and
// advance for it.
template <class C, class W>
__device__ __forceinline__ void copy_tiles(const AttnParams &P, const CUtensorMap &tmK, const CUtensorMap &tmV, W w, long long t1,
                                           int stop, uint32_t base, float *sc, uint32_t full, uint32_t empty, int lane) {
    const int pages = TILE / P.page;  // of a tile
    const uint32_t box = static_cast<uint32_t>(P.page) * C::ROW;
    int it = 0;
    bool ok = true;
    while (ok && w.t < t1) {
        const Span u = span_of<C::R>(P, w, t1);
        const int32_t *tab = P.table + static_cast<int64_t>(w.b) * P.ld_table;
        auto page_of = [&](int j) {  // of lane's page of tile j, -1 where there is nothing to read
            const int tok = u.from + j * TILE + lane * P.page;
            int id = -1;
            if (lane < pages && j < u.je && tok < u.hi && tok + P.page > u.lo) {
                id = __ldg(tab + tok / P.page);
                if (id < 0 || id >= P.pages) {
                    atomicOr(P.status, STATUS_INDEX);
                    id = -1;
                }
            }
            return id;
        };
        int id = page_of(u.jb);
        bool far = false;  // a value scale of the unit, up to here, is far from 1
        for (int j = u.jb; j < u.je; ++j, ++it) {
            const int64_t tile = static_cast<int64_t>(max(id, 0)) * P.heads + u.head;
            const float ks = __ldg(P.scales[0] + tile), vs = __ldg(P.scales[1] + tile);
            const int next = page_of(j + 1);
            const int s = it % C::STAGES;
            if (it >= stop) ok = false;
            if (ok && it >= C::STAGES) ok = __all_sync(0xffffffffu, mbar_wait(empty + 8 * s, ((it / C::STAGES) - 1) & 1, P.status));
            if (!ok) break;
            const int src = 16 * lane / P.page;  // scales of the groups of 16 tokens
            const float kg = __shfl_sync(0xffffffffu, ks, src), vg = __shfl_sync(0xffffffffu, vs, src);
            far = far || __any_sync(0xffffffffu, id >= 0 && far_scale(vs));
            if (lane < 8) {
                const float v = fmaxf(vg, 0x1p-100f);
                float *const d = sc + SCALES * s + lane;
                d[0] = kg, d[8] = log2f(v), d[16] = far ? 0.0f : __fdiv_rn(1.0f, v);
            }
            __syncwarp();  // (lane 0's arrival hands over what the eight wrote; a vote orders no memory)
            const uint32_t live = __popc(__ballot_sync(0xffffffffu, id >= 0));
            if (lane == 0) mbar_arrive_expect_tx(full + 8 * s, 2 * C::COLS * live * box);
            __syncwarp();
            if (id >= 0) {
                const uint32_t dst = base + s * C::STAGE + lane * box;
#pragma unroll
                for (int k = 0; k < C::COLS; ++k) {
                    tma_page(dst + k * TILE * 128, &tmK, 128 * k, static_cast<int>(tile), full + 8 * s);
                    tma_page(dst + C::SIDE + k * TILE * 128, &tmV, 128 * k, static_cast<int>(tile), full + 8 * s);
                }
            }
            id = next;
        }
        advance<C::R>(P, w, u.nt, t1);
    }
    // no CTA ends with copies in flight
    for (int i = max(0, it - C::STAGES); i < it; ++i) mbar_wait(full + 8 * (i % C::STAGES), (i / C::STAGES) & 1, P.status);
}

// The number of parts of a unit that were there before this CTA's, by one thread behind a
// barrier of those that wrote it: the fence carries their writes too.  (By all of them it
// took 1200 cycles, and 6600 where the others read at full rate.)  The last one, with `last`
// before it, leaves the counter zero for the next launch.  In the upper half of the counter and of
// what is returned: how many of the parts, this one included, have a value scale far from 1.
constexpr unsigned FAR_PART = 0x10000u;
__device__ __forceinline__ unsigned arrive(unsigned *count, unsigned last, bool far) {
    __threadfence();
    const unsigned mine = far ? FAR_PART : 0u, before = atomicAdd(count, 1u + mine);
    if ((before & (FAR_PART - 1)) == last) *count = 0u;
    __threadfence();
    return before + mine;
}

// The parts of a unit, of the CTAs c0 .. c1, joined in their order, eight at a time on
// their way; out(r, at, row) says where row r goes.  far: value scales may be so far apart
// that a sum over small ones fades beside the reference of large ones.
template <class C, int DP, class Out>
__device__ __forceinline__ void join_parts(const AttnParams &P, int c0, int c1, int rows, int tid, bool far, const Out &out) {
    for (int i = tid; i < rows * (DP / 4); i += C::CONSUMERS) {
        const int r = i / (DP / 4), d = 4 * (i % (DP / 4));
        float top = -INFINITY, sum = 0.0f;
        float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int k0 = c0; k0 <= c1; k0 += 8) {
            float pm[8], pl[8];
            float4 pv[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int cc = min(k0 + k, c1);
                const float *q = P.part + (static_cast<int64_t>(cc) * 2 + (cc == c0)) * C::PART;
                pm[k] = __ldcg(q + C::R * DP + r);
                pl[k] = __ldcg(q + C::R * (DP + 1) + r);
                pv[k] = __ldcg(reinterpret_cast<const float4 *>(q + r * DP + d));
            }
            float now = top;
#pragma unroll
            for (int k = 0; k < 8; ++k) now = fmaxf(now, pm[k]);
            const float ref = now == -INFINITY ? 0.0f : now, down = ex2(top - ref);
            top = now;
            sum *= down, y.x *= down, y.y *= down, y.z *= down, y.w *= down;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float f = k0 + k <= c1 ? ex2(pm[k] - ref) : 0.0f;
                if (k0 + k <= c1) {
                    sum = fmaf(pl[k], f, sum);
                    y.x = fmaf(pv[k].x, f, y.x), y.y = fmaf(pv[k].y, f, y.y);
                    y.z = fmaf(pv[k].z, f, y.z), y.w = fmaf(pv[k].w, f, y.w);
                }
            }
        }
        if (far) {
            sum = 0.0f;
#pragma unroll 1
            for (int cc = c0; cc <= c1; ++cc) {
                const float *q = P.part + (static_cast<int64_t>(cc) * 2 + (cc == c0)) * C::PART;
                sum += faded(__ldcg(q + C::R * (DP + 1) + r), __ldcg(q + C::R * DP + r) - (top == -INFINITY ? 0.0f : top));
            }
        }
        const float inv = sum != 0.0f ? L_FACTOR / sum : 0.0f;
        int64_t at, row;
        out(r, at, row);
        if (d < P.dim) {
            store_typed(P.y, at + d, P.y_type, y.x * inv);
            store_typed(P.y, at + d + 1, P.y_type, y.y * inv);
            store_typed(P.y, at + d + 2, P.y_type, y.z * inv);
            store_typed(P.y, at + d + 3, P.y_type, y.w * inv);
        }
        if (P.lse && d == 0) P.lse[row] = sum != 0.0f ? (top + log2f(sum) + 20.0f - C::SHIFT) * LN2 : -INFINITY;
    }
}

// The share of tokens tok and tok + 8 of two rows' sums (far_scale); x: their products, token by
// token; row: the rows' factors, R on the first tokens that they see, and so on.
template <class C, bool HL>
__device__ __forceinline__ void far_tokens(FarSum *apart, float4 x, float scale, int tok, const float *row) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int *const seen = reinterpret_cast<const int *>(row) + h;
        const int lo = seen[C::R], hi = seen[2 * C::R];
        const float f = row[h] * scale, low = HL ? row[3 * C::R + h] * scale : 0.0f;
        apart[h].add(2, L_FACTOR * 0x1p14f, [&](int i) {
            const float v = i ? (h ? x.w : x.z) : (h ? x.y : x.x);
            const int k = tok + 8 * i;
            return k >= lo && k < hi ? fmaf(v, f, v * low) : -INFINITY;
        });
    }
}

// The same as a function that is called: for four groups of rows what it takes of the registers
// costs more (8 sequences of 1024 tokens, 6 rows: 24.6 against 25.6 us; for fewer 17.9 against 16.9).
template <class C, bool HL>
__device__ __noinline__ void far_tokens_called(FarSum *apart, float4 x, float scale, int tok, const float *row) {
    far_tokens<C, HL>(apart, x, scale, tok, row);
}

template <int DP, int NB, bool HL>
__global__ void __launch_bounds__(THREADS + 32, Few<DP, NB, HL>::CTAS)
    kv_attention_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const AttnParams P) {
    using C = Few<DP, NB, HL>;
    constexpr int R = C::R, STAGES = C::STAGES, KS = DP / 16;
    constexpr int MT = DP / 16 >= 8 ? DP / 128 : 1;  // groups of 16 dims per warp
    constexpr int HALVES = DP == 64 ? 2 : 1;          // warps that share a group of dims, each with its tokens
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = smem_u32(smem);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31, g = lane >> 2, c = lane & 3;
    __half *const sq = reinterpret_cast<__half *>(smem + C::OFF_Q);
    __half *const sp = reinterpret_cast<__half *>(smem + C::OFF_P);
    float *const red = reinterpret_cast<float *>(smem + C::OFF_RED);
    float *const row_f = reinterpret_cast<float *>(smem + C::OFF_ROW);
    int *const row_lo = reinterpret_cast<int *>(row_f + R), *const row_hi = row_lo + R;
    float *const sc = reinterpret_cast<float *>(smem + C::OFF_SC);
    const uint32_t full = base + C::OFF_BAR, empty = full + 8 * STAGES;
    volatile unsigned *const arrived = reinterpret_cast<volatile unsigned *>(smem + C::OFF_BAR + 16 * STAGES);
    volatile unsigned *const some_nan = arrived + 1;  // a NaN among values that not all rows see, in some unit up to here

    if (tid == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 8);
        }
        fence_mbar_init();
        *some_nan = 0;
    }
    pdl_wait();
    pdl_trigger();

    Walk w;
    long long t1, W;
    int blocks;
    if (!begin_walk<R>(P, lane, w, t1, W, blocks)) return;
    __syncthreads();  // (the barriers are ready)

    if (warp == 8) {
        copy_tiles<C>(P, tmK, tmV, w, t1, blockIdx.x == 0 ? P.stop : NO_STOP, base, sc, full, empty, lane);
        return;
    }

    int it = 0;
    while (w.t < t1) {
        const Span u = span_of<R>(P, w, t1);
        const Seq &s = w.s;
        const int r0 = u.r0, rows = u.rows, head = u.head, start = s.len - s.n;

        // queries: one warp per row, times a power of two that brings the largest to [2^13, 2^14)
        // (the last unit's barriers lie between its reading of them and this)
        QueryRaw<HL> raw[NB][DP / 32];
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            const int qr = r0 + min(warp + 8 * n, rows - 1), i = token_of(P, qr);
            const int64_t at = (static_cast<int64_t>(s.row0) + i) * P.ldq_t + static_cast<int64_t>(head * P.group + (qr - i * P.group)) * P.ldq_h;
#pragma unroll
            for (int k = 0; k < DP / 32; ++k) raw[n][k] = __ldg(static_cast<const QueryRaw<HL> *>(P.q) + at + min(lane + 32 * k, P.dim - 1));
        }
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            const int r = warp + 8 * n, i = token_of(P, r0 + min(r, rows - 1));
            float v[DP / 32], top = 0.0f;
#pragma unroll
            for (int k = 0; k < DP / 32; ++k) {
                v[k] = r >= rows || lane + 32 * k >= P.dim ? 0.0f : query_value(raw[n][k], P.q_type);
                const float a = fabsf(v[k]);
                top = a <= 3.402823466e38f ? fmaxf(top, a) : top;
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            // (a power of two below 2^127 either way; tiny rows keep what fp32 holds of them)
            const int e = top > 0.0f ? min(max(13 - exponent_of(__float_as_uint(top)), -114), 100) : 0;
            const float up = pow2f(e);
#pragma unroll
            for (int k = 0; k < DP / 32; ++k) {
                const float x = v[k] * up + (v[k] - v[k]);  // (an infinity as NaN: its scores may all be -inf, as if nothing was seen)
                const __half h = __float2half_rn(x);
                sq[r * C::QP + lane + 32 * k] = h;
                if constexpr (HL) sq[(R + r) * C::QP + lane + 32 * k] = __float2half_rn(x - __half2float(h));
            }
            if (lane == 0) {
                row_f[r] = P.factor * pow2f(-e);
                if constexpr (HL) row_f[3 * R + r] = P.factor_low * pow2f(-e);
                row_hi[r] = P.causal ? min(s.len, start + i + 1) : s.len;
                row_lo[r] = seen_from(P, start + i);
            }
        }
        named_barrier(1, THREADS);
        // one group of rows in one part: its fragments stay in registers
        constexpr bool KEEP = NB == 1 && !HL && DP <= 128;
        uint2 qf[KEEP ? KS : 1];
        if constexpr (KEEP) {
#pragma unroll
            for (int k = 0; k < KS; ++k) qf[k] = *reinterpret_cast<const uint2 *>(sq + g * C::QP + 16 * k + 4 * c);
        }

        float o[MT][NB][4];
        float m[NB][2], l[NB][2];
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.0f;
#pragma unroll
            for (int k = 0; k < MT; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[k][n][i] = 0.0f;
        }

        FarSum apart[NB][2];
        bool far = false;
        for (int j = u.jb; j < u.je; ++j, ++it) {
            const int slot = it % STAGES;
            const bool ok = __all_sync(0xffffffffu, mbar_wait(full + 8 * slot, (it / STAGES) & 1, P.status));
            const uint32_t sk = base + slot * C::STAGE, sv = sk + C::SIDE;
            const int tok0 = s.lo + j * TILE;
            const bool whole = tok0 >= u.all_lo && tok0 + TILE <= u.all_hi;
            if (ok && !whole) {
                // What no row sees may be anything, a page that nobody sees is not even
                // there: P of them is 0, and so are their values from here on.  A token
                // that some rows see and some do not: spread_nans.
#pragma unroll 1
                for (int i = 0; i < 16 * KS / 32; ++i) {
                    const int row = 16 * warp + (32 * i + lane) / KS;
                    uint4 *v = reinterpret_cast<uint4 *>(smem + slot * C::STAGE + C::SIDE + C::at(row, (32 * i + lane) % KS));
                    const bool seen = tok0 + row >= u.lo && tok0 + row < u.hi, bad = seen && has_nan(*v);
                    if (!seen) *v = make_uint4(0, 0, 0, 0);
                    if (bad) *v = without_nan(*v), *some_nan = 1;
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // (before the next copy into the slot)
            }

            // S^T of this warp's 16 tokens
            float x[NB][4];
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) x[n][i] = 0.0f;
            {
                const int row = 16 * warp + (lane & 15);
#pragma unroll
                for (int k = 0; k < KS; k += 2) {
                    uint32_t f[4];
                    ldsm4(sk + C::at(row, k + (lane >> 4)), f);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t a[4] = {halves(f[2 * h]), halves(f[2 * h + 1]), halves_hi(f[2 * h]), halves_hi(f[2 * h + 1])};
#pragma unroll
                        for (int n = 0; n < NB; ++n) {
                            if constexpr (KEEP) {
                                mma16816(x[n], a, qf[k + h].x, qf[k + h].y);
                            } else {
                                const uint2 q = *reinterpret_cast<const uint2 *>(sq + (8 * n + g) * C::QP + 16 * (k + h) + 4 * c);
                                mma16816(x[n], a, q.x, q.y);
                            }
                            if constexpr (HL) {
                                const uint2 ql =
                                    *reinterpret_cast<const uint2 *>(sq + (R + 8 * n + g) * C::QP + 16 * (k + h) + 4 * c);
                                mma16816(x[n], a, ql.x, ql.y);
                            }
                        }
                    }
                }
            }
            const int tok = tok0 + 16 * warp + g;  // this lane's tokens: tok, tok + 8
            const float *const scales = sc + SCALES * slot + warp;
            const float ks = scales[0], lv = scales[8], iv = scales[16];
            if (iv == 0.0f) {  // the sums apart (far_scale)
#pragma unroll
                for (int n = 0; n < NB; ++n) {
                    const int r = 8 * n + 2 * c;
                    if (!far) apart[n][0].m = m[n][0], apart[n][0].l = l[n][0], apart[n][1].m = m[n][1], apart[n][1].l = l[n][1];
                    const float4 products = make_float4(x[n][0], x[n][1], x[n][2], x[n][3]);
                    if constexpr (NB == 4 && DP <= 128) far_tokens_called<C, HL>(apart[n], products, ks, tok, row_f + r);
                    else far_tokens<C, HL>(apart[n], products, ks, tok, row_f + r);
                }
                far = true;
            }
            uint32_t hidden = 0;  // bit 4 n + i: x[n][i] is masked
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                const int r = 8 * n + 2 * c;
                const float2 f = *reinterpret_cast<const float2 *>(row_f + r);
                const float f0 = f.x * ks, f1 = f.y * ks;
                float y[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] = fmaf(x[n][i], i & 1 ? f1 : f0, lv);
                if (!whole) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int k = tok + (i >> 1) * 8, rr = r + (i & 1);
                        if (k < row_lo[rr] || k >= row_hi[rr]) y[i] = -INFINITY, hidden |= 1u << (4 * n + i);
                    }
                }
                if constexpr (!HL) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[n][i] = y[i];
                }
                float a = fmaxf(y[0], y[2]), d = fmaxf(y[1], y[3]);
#pragma unroll
                for (int k = 4; k < 32; k <<= 1) {
                    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, k));
                    d = fmaxf(d, __shfl_xor_sync(0xffffffffu, d, k));
                }
                if (g == 0) *reinterpret_cast<float2 *>(red + warp * R + r) = make_float2(a, d);
            }
            if (named_barrier_or(1, THREADS, !ok)) return;  // (a wait ran out: nothing more of this CTA)
            float alpha[NB][2];
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                const int r = 8 * n + 2 * c;
                float2 top = make_float2(m[n][0], m[n][1]);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float2 v = *reinterpret_cast<const float2 *>(red + k * R + r);
                    top.x = fmaxf(top.x, v.x), top.y = fmaxf(top.y, v.y);
                }
                // For fp32 the reference is a whole number: log2 of the value scales is
                // one too, so its difference to x has no error of its own.  Otherwise it
                // is the maximum, whose p then is exact in fp16.
                if constexpr (HL) top.x = ceilf(top.x), top.y = ceilf(top.y);
                // (a row that has seen nothing yet: any finite reference)
                const float m0 = top.x == -INFINITY ? 0.0f : top.x, m1 = top.y == -INFINITY ? 0.0f : top.y;
                alpha[n][0] = ex2(m[n][0] - m0), alpha[n][1] = ex2(m[n][1] - m1);
                m[n][0] = top.x, m[n][1] = top.y;
                float p[4];
                if constexpr (HL) {
                    // fp32 in, fp32 out: one rounding from the product to the exponent
                    const float f0 = row_f[r] * ks, f1 = row_f[r + 1] * ks;
                    const float e0 = row_f[3 * R + r] * ks, e1 = row_f[3 * R + r + 1] * ks;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float d = fmaf(x[n][i], i & 1 ? e1 : e0, lv - (i & 1 ? m1 : m0));
                        p[i] = hidden >> (4 * n + i) & 1 ? 0.0f : ex2(fmaf(x[n][i], i & 1 ? f1 : f0, d)) * 0x1p14f;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) p[i] = ex2(x[n][i] - (i & 1 ? m1 : m0) + P_SHIFT);
                }
                l[n][0] = fmaf((p[0] + p[2]) * L_FACTOR, iv, l[n][0] * alpha[n][0]);
                l[n][1] = fmaf((p[1] + p[3]) * L_FACTOR, iv, l[n][1] * alpha[n][1]);
                // to shared memory, the tokens of a group of 16 in the order of
                // the second product's fragments: token 2 c' + 8 h + i at 4 c' + 2 h + i
                const int at = 16 * warp + 4 * (g >> 1) + (g & 1);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const __half h = __float2half_rn(p[i]);
                    __half *d = sp + (r + (i & 1)) * C::PP + at + (i >> 1) * 2;
                    *d = h;
                    if constexpr (HL) d[R * C::PP] = __float2half_rn(p[i] - __half2float(h));
                }
            }
            named_barrier(1, THREADS);
            // O^T += V^T P^T; for fp32 a tile's products are summed apart and added
            // with a rounding to nearest (the tensor cores cut off what an addition loses)
            const int wd = HALVES == 2 ? warp & 3 : warp, wt = HALVES == 2 ? warp >> 2 : 0;
            float part[HL ? MT : 1][HL ? NB : 1][4];
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int k = 0; k < MT; ++k)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if constexpr (HL) part[k][n][i] = 0.0f;
                        else o[k][n][i] *= alpha[n][i & 1];
                    }
            constexpr int KT = TILE / 16 / HALVES;
#pragma unroll
            for (int k = 0; k < KT; k += 2) {
                const int t16 = wt * KT + k;
                const int row = 16 * t16 + lane;
                uint2 pb[2][NB][C::PARTS];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int n = 0; n < NB; ++n)
#pragma unroll
                        for (int q = 0; q < C::PARTS; ++q)
                            pb[h][n][q] = *reinterpret_cast<const uint2 *>(sp + (q * R + 8 * n + g) * C::PP + 16 * (t16 + h) + 4 * c);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    uint32_t f[4];
                    ldsm4_t(sv + C::at(row, wd * MT + mt), f);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t u0 = __byte_perm(f[2 * h], 0, 0x3120), u1 = __byte_perm(f[2 * h + 1], 0, 0x3120);
                        const uint32_t a[4] = {halves(u0), halves_hi(u0), halves(u1), halves_hi(u1)};
#pragma unroll
                        for (int n = 0; n < NB; ++n)
#pragma unroll
                            for (int q = 0; q < C::PARTS; ++q) {
                                if constexpr (HL) mma16816(part[mt][n], a, pb[h][n][q].x, pb[h][n][q].y);
                                else mma16816(o[mt][n], a, pb[h][n][q].x, pb[h][n][q].y);
                            }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty + 8 * slot);
            if constexpr (HL) {
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int k = 0; k < MT; ++k)
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[k][n][i] = fmaf(o[k][n][i], alpha[n][i & 1], part[k][n][i]);
            }
        }
        named_barrier(1, THREADS);
        const bool nans = *some_nan != 0;  // (the same for all warps: none is past the next barrier)

        // sums over the lanes and warps that share a row
        if (far) {
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h) l[n][h] = apart[n][h].at(m[n][h]);
        }
#pragma unroll
        for (int n = 0; n < NB; ++n) {
#pragma unroll
            for (int k = 4; k < 32; k <<= 1) {
                l[n][0] += __shfl_xor_sync(0xffffffffu, l[n][0], k);
                l[n][1] += __shfl_xor_sync(0xffffffffu, l[n][1], k);
            }
            if (g == 0) *reinterpret_cast<float2 *>(red + warp * R + 8 * n + 2 * c) = make_float2(l[n][0], l[n][1]);
        }
        float *const half_o = reinterpret_cast<float *>(sp);  // (the probabilities are used up)
        static_assert(HALVES == 1 || 4 * NB * 4 * 32 * 4 <= C::PARTS * R * C::PP * 2, "half of the sums");
        if constexpr (HALVES == 2) {
            if (warp >= 4) {
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) half_o[((warp - 4) * NB * 4 + n * 4 + i) * 32 + lane] = o[0][n][i];
            }
        }
        named_barrier(1, THREADS);
        if constexpr (HALVES == 2) {
            if (warp < 4) {
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[0][n][i] += half_o[(warp * NB * 4 + n * 4 + i) * 32 + lane];
            }
        }
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            l[n][0] = l[n][1] = 0.0f;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float2 v = *reinterpret_cast<const float2 *>(red + k * R + 8 * n + 2 * c);
                l[n][0] += v.x, l[n][1] += v.y;
            }
        }

        auto out = [&](int r, int64_t &at, int64_t &row) {
            const int i = token_of(P, r0 + r), h = head * P.group + (r0 + r - i * P.group);
            at = (static_cast<int64_t>(s.row0) + i) * P.ldy_t + static_cast<int64_t>(h) * P.ldy_h;
            row = (static_cast<int64_t>(s.row0) + i) * P.heads * P.group + h;
        };
        const bool entire = u.nt == s.tiles;
        // (an entire unit's results, or a part of it: [row][dim] sums relative to m, then m and l)
        float *const mine = P.part + (static_cast<int64_t>(blockIdx.x) * 2 + (w.tile == 0)) * C::PART;
        if (entire) {
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = 8 * n + 2 * c + h;
                    if (r >= rows) continue;
                    int64_t at, row;
                    out(r, at, row);
                    const float inv = l[n][h] != 0.0f ? L_FACTOR / l[n][h] : 0.0f;
                    if (HALVES == 1 || warp < 4) {
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) {
                            const int d = 16 * (warp * MT + mt) + 2 * g;
                            if (d < P.dim) {
                                store_typed(P.y, at + d, P.y_type, o[mt][n][h] * inv);
                                store_typed(P.y, at + d + 1, P.y_type, o[mt][n][2 + h] * inv);
                            }
                        }
                    }
                    if (P.lse && warp == 0 && g == 0) P.lse[row] = l[n][h] != 0.0f ? (m[n][h] + log2f(l[n][h]) + 20.0f - C::SHIFT) * LN2 : -INFINITY;
                }
        } else {
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = 8 * n + 2 * c + h;
                    if (r >= rows) continue;
                    if (HALVES == 1 || warp < 4) {
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) {
                            const int d = 16 * (warp * MT + mt) + 2 * g;
                            *reinterpret_cast<float2 *>(mine + r * DP + d) = make_float2(o[mt][n][h], o[mt][n][2 + h]);
                        }
                    }
                    if (warp == 0 && g == 0) mine[R * DP + r] = m[n][h], mine[R * DP + R + r] = l[n][h];
                }
        }
        if (nans) {
            named_barrier(1, THREADS);
            spread_nans(P, w.b, head, start, r0, 0, rows, 0, DP, max(u.from + u.jb * TILE, u.lo), min(u.from + u.je * TILE, u.hi), u.all_lo,
                        u.all_hi, tid, THREADS, [&](int r, int d) {
                            int64_t at, row;
                            out(r, at, row);
                            if (entire) store_typed(P.y, at + d, P.y_type, __uint_as_float(A_NAN));
                            else mine[r * DP + d] = __uint_as_float(A_NAN);
                        });
        }
        if (!entire) {
            named_barrier(1, THREADS);
            const long long u0 = w.seq0 + w.unit * s.tiles, u1 = u0 + s.tiles - 1;  // first and last tile of the unit
            const int c0 = static_cast<int>(divide((u0 + 1) * blocks - 1, W)), c1 = static_cast<int>(divide((u1 + 1) * blocks - 1, W));
            if (tid == 0) *arrived = arrive(P.count + c0, static_cast<unsigned>(c1 - c0), far);
            named_barrier(1, THREADS);
            const unsigned parts = *arrived;
            if ((parts & (FAR_PART - 1)) == static_cast<unsigned>(c1 - c0)) join_parts<C, DP>(P, c0, c1, rows, tid, parts >= FAR_PART, out);
        }
        advance<R>(P, w, u.nt, t1);
    }
}

// The tensor map of codes [pages * heads][page][dim], boxes of a page and `cols` bytes.
inline bool encode_pages(CUtensorMap *m, const uint8_t *codes, const AttnParams &p, int cols) {
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(p.dim), static_cast<cuuint64_t>(p.page),
                                static_cast<cuuint64_t>(p.pages * p.heads)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(p.dim), static_cast<cuuint64_t>(p.dim) * p.page};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(cols), static_cast<cuuint32_t>(p.page), 1}, es[3] = {1, 1, 1};
    return tensor_map_encoder()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t *>(codes), dims, strides, box, es,
                                CU_TENSOR_MAP_INTERLEAVE_NONE, cols == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// One instance (a translation unit of its own per DP, as they take long to compile).
template <int DP, int NB, bool HL>
cudaError_t launch_few(const AttnParams &p, cudaStream_t st, int num_sms, int dev) {
    using C = Few<DP, NB, HL>;
    const auto kern = kv_attention_kernel<DP, NB, HL>;
    static OncePerDevice ready;
    const cudaError_t e = ready(dev, [&] { return set_smem_attrs(kern, C::SMEM); });
    if (e != cudaSuccess) return e;
    CUtensorMap tk = {}, tv = {};
    if (!encode_pages(&tk, p.codes[0], p, C::ROW) || !encode_pages(&tv, p.codes[1], p, C::ROW)) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(num_sms * C::CTAS));
    cfg.blockDim = dim3(THREADS + 32);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, tk, tv, p);
}
template <int DP>
cudaError_t launch_few_dp(const AttnParams &p, int nb, bool hl, cudaStream_t st, int num_sms, int dev) {
    if (nb == 1) return hl ? launch_few<DP, 1, true>(p, st, num_sms, dev) : launch_few<DP, 1, false>(p, st, num_sms, dev);
    if (nb == 2) return hl ? launch_few<DP, 2, true>(p, st, num_sms, dev) : launch_few<DP, 2, false>(p, st, num_sms, dev);
    return hl ? launch_few<DP, 4, true>(p, st, num_sms, dev) : launch_few<DP, 4, false>(p, st, num_sms, dev);
}
// The kernel for many rows (kv_attention_tc.cu): 16-bit queries, heads of up to
// 128 values; cudaErrorNotSupported where the build gave it too few registers.
size_t tc_part_bytes(int dim, int num_sms);
cudaError_t launch_tc(const AttnParams &a, cudaStream_t st, int num_sms, int dev);
// The kernel for few 16-bit rows, at most 32 of a sequence and cache head on the average (kv_attention_slim.cu).
cudaError_t launch_slim(const AttnParams &a, int rows, cudaStream_t st, int num_sms, int dev);
// The kernel for many fp32 rows (kv_attention_rows.cu).
size_t rows_part_bytes(int dim, int num_sms);
cudaError_t launch_rows(const AttnParams &a, cudaStream_t st, int num_sms, int dev);

cudaError_t launch_few_64(const AttnParams &p, int nb, bool hl, cudaStream_t st, int num_sms, int dev);
cudaError_t launch_few_128(const AttnParams &p, int nb, bool hl, cudaStream_t st, int num_sms, int dev);
cudaError_t launch_few_256(const AttnParams &p, int nb, bool hl, cudaStream_t st, int num_sms, int dev);

}  // namespace kv
}  // namespace qk
