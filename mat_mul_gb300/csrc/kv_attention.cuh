// kv_attention.cuh -- attention over the paged 8-bit cache for few query rows
// per cache head (decode, drafted tokens) and for fp32 queries: one pass over
// the cache on mma.sync, work cut along the tokens and joined.
//
//   y = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q.k_j),  k_j = sk code, v_j = sv code,
// with one scale sk, sv per page and head.  A row's scores in powers of two,
//   x_j = (scale log2 e) sk (q.code_j) + log2 sv,  m = max x_j,  p'_j = 2^(x_j - m),
// carry the scale of the values: the second product then takes codes, y =
// sum p' code / sum (p' / sv), and p' <= 1 whatever the scales are.
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
// has to add up accumulators but across cut units.
#pragma once

#include "kv_device.cuh"
#include "qmm_internal.h"

namespace qk {

namespace kv {

constexpr int TILE = 128;     // tokens of a tile
constexpr int THREADS = 256;  // 8 warps
constexpr int LEAST = 2;      // tiles per block below which fewer blocks take part

// A power of two on p', so that its low part in fp16 keeps 2^-38 of the largest.
constexpr float P_SHIFT = 14.0f;
// and one on the sum of p' / sv, which then stays within fp32 for 2^31 tokens
// of any scale from 2^-100 to 2^120
constexpr float L_FACTOR = 0x1p-20f;

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
    float *lse;
    float *part;
    unsigned *count;
    int *status;
};

// A sequence of the batch and its share of the work: `units` = heads x row
// blocks, each of `tiles` tiles from token lo (a multiple of TILE) on.
struct Seq {
    int row0, n, len, lo, tiles, blocks;
    int64_t units;
};

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
    s.lo = 0;
    if (P.window) s.lo = max(0, len - s.n - P.window + 1) & ~(TILE - 1);
    s.tiles = max(1, (len - s.lo + TILE - 1) / TILE);
    const int64_t blocks = (static_cast<int64_t>(s.n) * P.group + R - 1) / R;
    s.blocks = static_cast<int>(blocks);
    s.units = blocks * P.heads;
    return true;
}

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool live) {
    const int n = live ? 16 : 0;  // the rest is filled with zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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

__device__ __forceinline__ float load_typed(const void *p, int64_t i, int type) {
    if (type == QMM_F32) return __ldg(static_cast<const float *>(p) + i);
    if (type == QMM_F16) return __half2float(__ldg(static_cast<const __half *>(p) + i));
    return __bfloat162float(__ldg(static_cast<const __nv_bfloat16 *>(p) + i));
}
__device__ __forceinline__ void store_typed(void *p, int64_t i, int type, float v) {
    if (type == QMM_F32) static_cast<float *>(p)[i] = v;
    else if (type == QMM_F16) static_cast<__half *>(p)[i] = __float2half_rn(v);
    else static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
}

// DP: dim rounded up to 64, 128 or 256; NB: groups of eight query rows of a
// block; HL: queries and probabilities as two fp16 parts.
template <int DP, int NB, bool HL>
struct Few {
    static constexpr int R = 8 * NB, PARTS = HL ? 2 : 1;
    static constexpr int STAGES = DP == 256 ? 2 : 3;
    static constexpr int SIDE = TILE * DP, STAGE = 2 * SIDE;
    static constexpr int QP = DP + 16, PP = TILE + 16;  // pitches in halves: 8 banks between rows, as 8-byte reads want
    static constexpr int OFF_Q = STAGES * STAGE;
    static constexpr int OFF_P = OFF_Q + PARTS * R * QP * 2;
    static constexpr int OFF_RED = OFF_P + PARTS * R * PP * 2;       // [8 warps][R]
    static constexpr int OFF_ROW = OFF_RED + 8 * R * 4;              // [R] factor of the row, [R] first, [R] end, [R] the factor's low part
    static constexpr int OFF_SC = OFF_ROW + 4 * R * 4;               // [STAGES][2][8] scales
    static constexpr int OFF_ID = OFF_SC + STAGES * 16 * 4;          // [STAGES + 1][8] page ids
    static constexpr int OFF_PRE = (OFF_ID + (STAGES + 1) * 8 * 4 + 7) / 8 * 8;  // prefix sums
    static constexpr int SMEM = OFF_PRE + (THREADS + 1) * 8 + 64;
    static constexpr int PART = R * (DP + 2);  // floats of a partial result
};

template <int DP, int NB, bool HL>
__global__ void __launch_bounds__(THREADS, DP == 256 ? 1 : 2) kv_attention_kernel(const AttnParams P) {
    using C = Few<DP, NB, HL>;
    constexpr int R = C::R, STAGES = C::STAGES, KS = DP / 16;
    constexpr int MT = DP / 16 >= 8 ? DP / 128 : 1;  // groups of 16 dims per warp
    constexpr int HALVES = DP == 64 ? 2 : 1;          // warps that share a group of dims, each with its tokens
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t base = smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    __half *const sq = reinterpret_cast<__half *>(smem + C::OFF_Q);
    __half *const sp = reinterpret_cast<__half *>(smem + C::OFF_P);
    float *const red = reinterpret_cast<float *>(smem + C::OFF_RED);
    float *const row_f = reinterpret_cast<float *>(smem + C::OFF_ROW);
    int *const row_lo = reinterpret_cast<int *>(row_f + R), *const row_hi = row_lo + R;
    const float *const sc = reinterpret_cast<const float *>(smem + C::OFF_SC);
    int *const ids = reinterpret_cast<int *>(smem + C::OFF_ID);
    long long *const pre = reinterpret_cast<long long *>(smem + C::OFF_PRE);
    __shared__ unsigned arrived;

    pdl_wait();
    pdl_trigger();

    // the tiles of the sequences before each thread's share of them
    const int share = (P.B + THREADS - 1) / THREADS;
    {
        long long sum = 0;
        for (int b = tid * share; b < min(P.B, (tid + 1) * share); ++b) {
            Seq s;
            if (!load_seq<R>(P, b, s)) atomicOr(P.status, STATUS_INDEX);
            sum += s.units * s.tiles;
        }
        long long incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) pre[warp] = incl;
        __syncthreads();
        long long before = 0;
        for (int w = 0; w < warp; ++w) before += pre[w];
        __syncthreads();
        pre[tid] = before + incl - sum;
        if (tid == THREADS - 1) pre[THREADS] = before + incl;
    }
    if (DP > P.dim) {  // the columns that no copy writes
        uint4 *z = reinterpret_cast<uint4 *>(smem);
        for (int i = tid; i < STAGES * C::STAGE / 16; i += THREADS) z[i] = make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
    const long long W = pre[THREADS];
    if (W == 0) return;
    const long long most = max(1ll, W / LEAST);
    const int blocks = static_cast<int>(min(static_cast<long long>(gridDim.x), most));
    const int cta = blockIdx.x;
    if (cta >= blocks) return;
    long long t = cta * W / blocks;
    const long long t1 = (cta + 1) * W / blocks;

    int b, tile;
    int64_t unit;
    Seq s;
    long long seq0;  // tiles before sequence b
    {
        int first = 0, last = THREADS - 1;
        while (first < last) {
            const int mid = (first + last + 1) >> 1;
            if (pre[mid] <= t) first = mid;
            else last = mid - 1;
        }
        b = first * share;
        seq0 = pre[first];
        for (;; ++b) {
            load_seq<R>(P, b, s);
            if (t < seq0 + s.units * s.tiles) break;
            seq0 += s.units * s.tiles;
        }
        unit = (t - seq0) / s.tiles;
        tile = static_cast<int>((t - seq0) - unit * s.tiles);
    }

    // copies: this thread's 16-byte column and rows of a tile
    constexpr int CPR = DP / 16, STEP = THREADS / CPR;
    const int my_c = tid % CPR, my_r = tid / CPR;
    const bool copies = my_c < P.dim / 16;
    auto swz = [](int row) { return DP == 64 ? (row >> 1) & 3 : row & 7; };

    while (t < t1) {
        const int head = static_cast<int>(unit / s.blocks), block = static_cast<int>(unit - static_cast<int64_t>(head) * s.blocks);
        const int nt = static_cast<int>(min(static_cast<long long>(s.tiles - tile), t1 - t));
        const int64_t r0 = static_cast<int64_t>(block) * R;
        const int rows = static_cast<int>(min(static_cast<int64_t>(R), static_cast<int64_t>(s.n) * P.group - r0));
        // tokens that some row of the block sees, and those that all of them see
        const int start = s.len - s.n;
        const int i0 = static_cast<int>(r0 / P.group), i1 = static_cast<int>((r0 + rows - 1) / P.group);
        const int hi = P.causal ? min(s.len, start + i1 + 1) : s.len;
        const int all_hi = P.causal ? min(s.len, start + i0 + 1) : s.len;
        const int lo = P.window ? max(0, start + i0 - P.window + 1) : 0;
        const int all_lo = P.window ? max(0, start + i1 - P.window + 1) : 0;
        const int jb = max(tile, (lo - s.lo) / TILE), je = min(tile + nt, hi > s.lo ? (hi - s.lo + TILE - 1) / TILE : 0);

        __syncthreads();  // nobody reads what the last segment left in shared memory
        const int32_t *ptab = P.table + static_cast<int64_t>(b) * P.ld_table;
        // ids of the eight groups of 16 tokens of tile j, -1 where there is nothing to read
        auto page_of = [&](int j) {
            const int tok = s.lo + j * TILE + 16 * tid;
            int id = -1;
            if (tid < 8 && j < je && tok < hi && tok + 15 >= lo) {
                id = __ldg(ptab + tok / P.page);
                if (id < 0 || id >= P.pages) {
                    atomicOr(P.status, STATUS_INDEX);
                    id = -1;
                }
            }
            return id;
        };
        auto copy_tile = [&](int j) {
            if (j < je) {
                const int slot = (j - jb) % STAGES;
                const int *id = ids + ((j - jb) % (STAGES + 1)) * 8;
                const uint32_t dst = base + slot * C::STAGE;
                const int tok0 = s.lo + j * TILE;
#pragma unroll
                for (int i = 0; i < TILE / STEP; ++i) {
                    const int r = my_r + i * STEP;
                    const int page = id[r >> 4];
                    const bool live = page >= 0 && tok0 + r < hi;
                    const int64_t at =
                        live ? ((static_cast<int64_t>(page) * P.heads + head) * P.page + ((tok0 + r) & (P.page - 1))) * P.dim + 16 * my_c
                             : 0;
                    const uint32_t d = dst + r * DP + ((my_c ^ swz(r)) << 4);
                    if (copies) {
                        cp16(d, P.codes[0] + at, live);
                        cp16(d + C::SIDE, P.codes[1] + at, live);
                    }
                }
                if (tid < 16) {
                    const int page = max(id[tid & 7], 0);
                    cp4(base + C::OFF_SC + (slot * 16 + tid) * 4, P.scales[tid >> 3] + static_cast<int64_t>(page) * P.heads + head);
                }
            }
            cp_commit();
        };
        if (tid < 8) {
#pragma unroll
            for (int j = 0; j < STAGES; ++j) ids[j * 8 + tid] = page_of(jb + j);
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < STAGES - 1; ++j) copy_tile(jb + j);

        // queries: one warp per row, times a power of two that brings the largest to [2^13, 2^14)
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            const int r = warp + 8 * n;
            float v[DP / 32];
            float top = 0.0f;
            const bool live = r < rows;
            const int64_t qr = r0 + (live ? r : 0);
            const int i = static_cast<int>(qr / P.group);
            const int64_t at = (s.row0 + i) * P.ldq_t + (head * P.group + (qr - static_cast<int64_t>(i) * P.group)) * P.ldq_h;
#pragma unroll
            for (int k = 0; k < DP / 32; ++k) {
                const int d = lane + 32 * k;
                v[k] = live && d < P.dim ? load_typed(P.q, at + d, P.q_type) : 0.0f;
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
                const float w = v[k] * up;
                const __half h = __float2half_rn(w);
                sq[r * C::QP + lane + 32 * k] = h;
                if constexpr (HL) sq[(R + r) * C::QP + lane + 32 * k] = __float2half_rn(w - __half2float(h));
            }
            if (lane == 0) {
                row_f[r] = P.factor * pow2f(-e);
                if constexpr (HL) row_f[3 * R + r] = P.factor_low * pow2f(-e);
                row_hi[r] = P.causal ? min(s.len, start + i + 1) : s.len;
                row_lo[r] = P.window ? start + i - P.window + 1 : 0;
            }
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

        for (int j = jb; j < je; ++j) {
            const int slot = (j - jb) % STAGES;
            cp_wait<STAGES - 2>();
            __syncthreads();
            copy_tile(j + STAGES - 1);
            const int next_id = page_of(j + STAGES);
            const uint32_t sk = base + slot * C::STAGE, sv = sk + C::SIDE;

            // S^T of this warp's 16 tokens
            float x[NB][4];
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) x[n][i] = 0.0f;
            {
                const int row = 16 * warp + (lane & 15);
                const uint32_t ra = sk + row * DP;
#pragma unroll
                for (int k = 0; k < KS; k += 2) {
                    uint32_t w[4];
                    ldsm4(ra + (((k + (lane >> 4)) ^ swz(row)) << 4), w);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t a[4] = {halves(w[2 * h]), halves(w[2 * h + 1]), halves_hi(w[2 * h]), halves_hi(w[2 * h + 1])};
#pragma unroll
                        for (int n = 0; n < NB; ++n) {
                            const uint2 q = *reinterpret_cast<const uint2 *>(sq + (8 * n + g) * C::QP + 16 * (k + h) + 4 * c);
                            mma16816(x[n], a, q.x, q.y);
                            if constexpr (HL) {
                                const uint2 ql =
                                    *reinterpret_cast<const uint2 *>(sq + (R + 8 * n + g) * C::QP + 16 * (k + h) + 4 * c);
                                mma16816(x[n], a, ql.x, ql.y);
                            }
                        }
                    }
                }
            }
            const int tok = s.lo + j * TILE + 16 * warp + g;  // this lane's tokens: tok, tok + 8
            const float ks = sc[slot * 16 + warp], vs = fmaxf(sc[slot * 16 + 8 + warp], 0x1p-100f);
            const float lv = log2f(vs), iv = __fdiv_rn(1.0f, vs);
            uint32_t hidden = 0;  // bit 4 n + i: x[n][i] is masked
            const bool whole = s.lo + j * TILE >= all_lo && s.lo + (j + 1) * TILE <= all_hi;
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                const int r = 8 * n + 2 * c;
                const float f0 = row_f[r] * ks, f1 = row_f[r + 1] * ks;
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
            __syncthreads();
            if (tid < 8) ids[((j + STAGES - jb) % (STAGES + 1)) * 8 + tid] = next_id;
            float alpha[NB][2];
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                const int r = 8 * n + 2 * c;
                float2 top = make_float2(m[n][0], m[n][1]);
#pragma unroll
                for (int w = 0; w < 8; ++w) {
                    const float2 v = *reinterpret_cast<const float2 *>(red + w * R + r);
                    top.x = fmaxf(top.x, v.x), top.y = fmaxf(top.y, v.y);
                }
                // The reference is a whole number: log2 of the value scales is one
                // too, so its difference to x has no error of its own.
                top.x = ceilf(top.x), top.y = ceilf(top.y);
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
            __syncthreads();
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
                    const int chunk = wd * MT + mt;
                    uint32_t w[4];
                    ldsm4_t(sv + row * DP + ((chunk ^ swz(row)) << 4), w);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t u0 = __byte_perm(w[2 * h], 0, 0x3120), u1 = __byte_perm(w[2 * h + 1], 0, 0x3120);
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
            if constexpr (HL) {
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int k = 0; k < MT; ++k)
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[k][n][i] = fmaf(o[k][n][i], alpha[n][i & 1], part[k][n][i]);
            }
        }
        cp_wait<0>();
        __syncthreads();

        // sums over the lanes and warps that share a row
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
        __syncthreads();
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
            for (int w = 0; w < 8; ++w) {
                const float2 v = *reinterpret_cast<const float2 *>(red + w * R + 8 * n + 2 * c);
                l[n][0] += v.x, l[n][1] += v.y;
            }
        }

        auto out = [&](int r, int64_t &at, int64_t &row) {
            const int64_t qr = r0 + r;
            const int i = static_cast<int>(qr / P.group);
            const int h = head * P.group + static_cast<int>(qr - static_cast<int64_t>(i) * P.group);
            at = (s.row0 + i) * P.ldy_t + h * P.ldy_h;
            row = (static_cast<int64_t>(s.row0) + i) * P.heads * P.group + h;
        };
        const bool cut = nt < s.tiles;
        if (!cut) {
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
                    if (P.lse && warp == 0 && g == 0)
                        P.lse[row] = l[n][h] != 0.0f ? (m[n][h] + log2f(l[n][h]) + 20.0f - P_SHIFT) * 0.6931471805599453f : -INFINITY;
                }
        } else {
            // a part of a unit: [row][dim] sums relative to m, then m and l
            float *const mine = P.part + (static_cast<int64_t>(cta) * 2 + (tile == 0)) * C::PART;
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
            __threadfence();
            __syncthreads();
            const long long u0 = seq0 + unit * s.tiles, u1 = u0 + s.tiles - 1;  // first and last tile of the unit
            const int c0 = static_cast<int>(((u0 + 1) * blocks - 1) / W), c1 = static_cast<int>(((u1 + 1) * blocks - 1) / W);
            if (tid == 0) arrived = atomicAdd(P.count + c0, 1u);
            __syncthreads();
            if (arrived == static_cast<unsigned>(c1 - c0)) {
                if (tid == 0) P.count[c0] = 0u;  // zero again for the next launch
                __threadfence();
                // the last one joins them, in their order
                for (int i = tid; i < rows * (DP / 4); i += THREADS) {
                    const int r = i / (DP / 4), d = 4 * (i % (DP / 4));
                    float top = -INFINITY;
                    for (int k = c0; k <= c1; ++k)
                        top = fmaxf(top, __ldcg(P.part + (static_cast<int64_t>(k) * 2 + (k == c0)) * C::PART + R * DP + r));
                    const float ref = top == -INFINITY ? 0.0f : top;
                    float sum = 0.0f;
                    float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    for (int k = c0; k <= c1; ++k) {
                        const float *q = P.part + (static_cast<int64_t>(k) * 2 + (k == c0)) * C::PART;
                        const float w = ex2(__ldcg(q + R * DP + r) - ref);
                        sum = fmaf(__ldcg(q + R * DP + R + r), w, sum);
                        const float4 v = __ldcg(reinterpret_cast<const float4 *>(q + r * DP + d));
                        y.x = fmaf(v.x, w, y.x), y.y = fmaf(v.y, w, y.y), y.z = fmaf(v.z, w, y.z), y.w = fmaf(v.w, w, y.w);
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
                    if (P.lse && d == 0) P.lse[row] = sum != 0.0f ? (top + log2f(sum) + 20.0f - P_SHIFT) * 0.6931471805599453f : -INFINITY;
                }
            }
        }

        // the next unit
        t += nt;
        tile = 0;
        if (t < t1 && ++unit == s.units) {
            seq0 += s.units * s.tiles;
            unit = 0;
            do load_seq<R>(P, ++b, s);
            while (s.units == 0);
        }
    }
}

// One instance (a translation unit of its own per DP, as they take long to compile).
template <int DP, int NB, bool HL>
cudaError_t launch_few(const AttnParams &p, cudaStream_t st, int num_sms, int dev) {
    using C = Few<DP, NB, HL>;
    const auto kern = kv_attention_kernel<DP, NB, HL>;
    static OncePerDevice ready;
    const cudaError_t e = ready(dev, [&] { return set_smem_attrs(kern, C::SMEM); });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(num_sms * (DP == 256 ? 1 : 2)));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}
template <int DP>
cudaError_t launch_few_dp(const AttnParams &p, int nb, bool hl, cudaStream_t st, int num_sms, int dev) {
    if (nb == 1) return hl ? launch_few<DP, 1, true>(p, st, num_sms, dev) : launch_few<DP, 1, false>(p, st, num_sms, dev);
    if (nb == 2) return hl ? launch_few<DP, 2, true>(p, st, num_sms, dev) : launch_few<DP, 2, false>(p, st, num_sms, dev);
    return hl ? launch_few<DP, 4, true>(p, st, num_sms, dev) : launch_few<DP, 4, false>(p, st, num_sms, dev);
}
// The kernel for many rows (kv_attention_tc.cu): 16-bit queries, heads of up to
// 128 values.  stop: the tile at which the first CTA's copies stop (NO_STOP: none).
size_t tc_part_bytes(int dim, int num_sms);
cudaError_t launch_tc(const AttnParams &a, int stop, cudaStream_t st, int num_sms, int dev);

cudaError_t launch_few_64(const AttnParams &p, int nb, bool hl, cudaStream_t st, int num_sms, int dev);
cudaError_t launch_few_128(const AttnParams &p, int nb, bool hl, cudaStream_t st, int num_sms, int dev);
cudaError_t launch_few_256(const AttnParams &p, int nb, bool hl, cudaStream_t st, int num_sms, int dev);

}  // namespace kv
}  // namespace qk
