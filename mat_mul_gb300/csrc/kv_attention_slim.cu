// kv_attention_slim.cu -- attention over the paged 8-bit cache for few fp16 or
// bf16 query rows per cache head (decode, drafted tokens), heads of up to 128 values.
//
// Formulas, sharing of the work and copies are those of kv_attention.cuh.  Here the
// query rows are the M side of both products and a warp takes 16 tokens of every
// tile for all of them:
//   S [16 MT rows x 16 tokens] = Q K^T      Q as fragments in shared memory
//   O [16 MT rows x dim]      += P V        P from the registers that held S
// so a warp has a maximum, a sum and an O of its own, nothing is exchanged and no
// warp waits for another until a unit ends; then the eight are joined through
// shared memory.
//
// fp16 rows keep the maximum as the reference, whose probability then is exact in
// fp16; bf16 rows move it only when it has grown by more than 2^8 of it.
//
// Measured (8 sequences of 16384 tokens, 5 rows of 32 heads, 8 heads of 128 in the
// cache): 95 us with fp16, 88 with bf16, 2.8 and 3.1 TB/s of codes (of 32 rows 20 are there);
// kv_attention.cuh's kernel, with two barriers a tile, 120 with fp16.  A tile takes 2000 cycles:
// 1024 of them products, 160 conversions, the rest one after another in two warps.
#include <type_traits>

#include "kv_attention.cuh"

namespace qk {
namespace kv {

namespace {

// Two warpgroups of consumers and one of which a warp brings the tiles; registers per
// thread at launch and after the split.
constexpr int SLIM_THREADS = THREADS + 128;
constexpr int REGS = 168, REGS_COPY = 56, REGS_MAIN = 224;
static_assert(128 * REGS_COPY + THREADS * REGS_MAIN <= SLIM_THREADS * REGS, "register split");

template <int DP, int MT>
struct Slim {
    static constexpr int R = 16 * MT, CONSUMERS = THREADS, STAGES = DP == 64 ? 7 : 4;
    static constexpr float SHIFT = 6.0f;  // P as fp16 is at most 2^(8 + SHIFT)
    static constexpr int ROW = DP == 64 ? 64 : 128, COLS = DP / ROW;
    static constexpr int SIDE = TILE * DP, STAGE = 2 * SIDE;
    static constexpr int OFF_Q = STAGES * STAGE;                    // [MT][DP / 16][lane] fragments
    static constexpr int SUM_ROW = DP + 16;                         // floats (banks of its own for the next row)
    static constexpr int OFF_SUM = OFF_Q + MT * DP / 16 * 512;      // [8 warps][16][SUM_ROW]
    static constexpr int OFF_ROW = OFF_SUM + 8 * 16 * SUM_ROW * 4;  // [R] factor, [R] first, [R] end, [R] reference, [R] sum
    static constexpr int OFF_WARP = OFF_ROW + 5 * R * 4;            // [8][R] references, [8][R] sums
    static constexpr int OFF_SC = OFF_WARP + 16 * R * 4;            // [STAGES] scales
    static constexpr int OFF_BAR = (OFF_SC + STAGES * SCALES * 4 + 7) / 8 * 8;
    static constexpr int SMEM = OFF_BAR + 16 * STAGES + 16;
    static_assert(SMEM <= 232448, "shared memory");
    static constexpr int PART = R * (DP + 2);
    static __device__ __forceinline__ int at(int row, int c) {
        if constexpr (DP == 64) return row * 64 + ((c ^ (row >> 1 & 3)) << 4);
        else return row * 128 + ((c ^ (row & 7)) << 4);
    }
};

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// 16 tokens' share of two rows' sums (far_scale), from scores of its own: a function that is
// called, so that in the ordinary case nothing of it takes a register.  row: the rows' factors, R on
// the first tokens that they see and 2 R on the ends of those.
template <class C>
__device__ __noinline__ void far_tile(FarSum *apart, uint32_t sk, const uint4 *my_q, float scale, int tok, const float *row) {
    float y[2][4] = {};
#pragma unroll 1
    for (int k = 0; k < C::SIDE / TILE / 16; k += 2) {
        uint32_t a[4];
        ldsm4(sk ^ (k << 4), a);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint4 q = my_q[32 * (k + h)];
            const uint32_t qa[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int n = 0; n < 2; ++n) mma16816(y[n], qa, halves(a[h + 2 * n]), halves_hi(a[h + 2 * n]));
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int *const seen = reinterpret_cast<const int *>(row) + 8 * h;
        const int lo = seen[C::R], hi = seen[2 * C::R];
        const float f = row[8 * h] * scale;
        apart[h].add(4, L_FACTOR * 0x1p6f, [&](int i) {
            const int k = tok + 8 * (i >> 1) + (i & 1);
            return k >= lo && k < hi ? y[i >> 1][2 * h + (i & 1)] * f : -INFINITY;
        });
    }
}

template <int DP, int MT>
__global__ void __launch_bounds__(SLIM_THREADS, 1)
    kv_attention_slim_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const AttnParams P) {
    using C = Slim<DP, MT>;
    constexpr int R = C::R, STAGES = C::STAGES, KS = DP / 16;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = smem_u32(smem);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31, g = lane >> 2, c = lane & 3;
    __half *const sq = reinterpret_cast<__half *>(smem + C::OFF_Q);
    float *const sums = reinterpret_cast<float *>(smem + C::OFF_SUM);
    float *const row_f = reinterpret_cast<float *>(smem + C::OFF_ROW);
    int *const row_lo = reinterpret_cast<int *>(row_f + R), *const row_hi = row_lo + R;
    float *const row_m = row_f + 3 * R, *const row_l = row_m + R;
    float *const warp_m = reinterpret_cast<float *>(smem + C::OFF_WARP), *const warp_l = warp_m + 8 * R;
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

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_COPY));
        if (warp == 8) copy_tiles<C>(P, tmK, tmV, w, t1, blockIdx.x == 0 ? P.stop : NO_STOP, base, sc, full, empty, lane);
        return;
    }
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_MAIN));

    const float move = P.q_type == QMM_F16 ? 0.0f : 8.0f;
    int it = 0;
    bool dead = false;  // a wait ran out: this warp only goes through the barriers from here on
    while (w.t < t1) {
        const Span u = span_of<R>(P, w, t1);
        const Seq &s = w.s;
        const int r0 = u.r0, rows = u.rows, head = u.head, start = s.len - s.n;

        // queries: one warp per row, times a power of two that brings the largest to [2^13, 2^14)
        // (the last unit's barriers lie between its reading of them and this)
        QueryRaw<false> raw[2 * MT][DP / 32];
#pragma unroll
        for (int n = 0; n < 2 * MT; ++n) {
            const int qr = r0 + min(warp + 8 * n, rows - 1), i = token_of(P, qr);
            const int64_t at = (static_cast<int64_t>(s.row0) + i) * P.ldq_t + static_cast<int64_t>(head * P.group + (qr - i * P.group)) * P.ldq_h;
#pragma unroll
            for (int k = 0; k < DP / 32; ++k) raw[n][k] = __ldg(static_cast<const QueryRaw<false> *>(P.q) + at + min(lane + 32 * k, P.dim - 1));
        }
#pragma unroll
        for (int n = 0; n < 2 * MT; ++n) {
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
            const int e = top > 0.0f ? min(max(13 - exponent_of(__float_as_uint(top)), -114), 100) : 0;
            const float up = pow2f(e);
#pragma unroll
            for (int k = 0; k < DP / 32; ++k) {
                // value d of row r: of fragment d / 16, lane 4 (r % 8) + d % 16 / 4, word 2 (d % 4 / 2) + r % 16 / 8
                const int d = lane + 32 * k;
                const float x = v[k] * up + (v[k] - v[k]);  // (an infinity as NaN)
                sq[(((n >> 1) * KS + (d >> 4)) * 32 + 4 * warp + (d >> 2 & 3)) * 8 + 4 * (d >> 1 & 1) + 2 * (n & 1) + (d & 1)] = __float2half_rn(x);
            }
            if (lane == 0) {
                row_f[r] = P.factor * pow2f(-e);
                row_hi[r] = P.causal ? min(s.len, start + i + 1) : s.len;
                row_lo[r] = seen_from(P, start + i);
            }
        }
        named_barrier(1, THREADS);
        const uint4 *const my_q = reinterpret_cast<const uint4 *>(sq) + lane;
        constexpr bool KEEP = MT == 1;  // fragments in registers
        uint4 qf[KEEP ? KS : 1];
        if constexpr (KEEP) {
#pragma unroll
            for (int k = 0; k < KS; ++k) qf[k] = my_q[32 * k];
        }
        float f[MT][2];
#pragma unroll
        for (int t = 0; t < MT; ++t) f[t][0] = row_f[16 * t + g], f[t][1] = row_f[16 * t + g + 8];

        float o[MT][DP / 8][4];
        float m[MT][2], l[MT][2];
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            m[t][0] = m[t][1] = -INFINITY;
            l[t][0] = l[t][1] = 0.0f;
#pragma unroll
            for (int n = 0; n < DP / 8; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[t][n][i] = 0.0f;
        }

        FarSum apart[MT][2];
        bool far = false;
        for (int j = u.jb; j < u.je; ++j, ++it) {
            const int slot = it % STAGES;
            if (!dead) dead = !__all_sync(0xffffffffu, mbar_wait(full + 8 * slot, (it / STAGES) & 1, P.status));
            // (a row's 16-byte chunks lie in the order of its swizzle: another chunk is an exclusive or away)
            const uint32_t sk = base + slot * C::STAGE + 16 * warp * C::ROW + C::at((lane & 7) + (lane >> 4 << 3), lane >> 3 & 1);
            const uint32_t sv = base + slot * C::STAGE + C::SIDE + 16 * warp * C::ROW + C::at(lane & 15, lane >> 4);
            const int from = u.from + j * TILE + 16 * warp;  // this warp's tokens
            if (!dead && from < u.hi && from + 16 > u.lo && sc[SCALES * slot + 16] == 0.0f) {  // the sums apart (far_scale)
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    if (!far) apart[t][0].m = m[t][0], apart[t][0].l = l[t][0], apart[t][1].m = m[t][1], apart[t][1].l = l[t][1];
                    far_tile<C>(apart[t], sk, my_q + 32 * KS * t, sc[SCALES * slot + warp], from + 2 * c, row_f + 16 * t + g);
                }
                far = true;
            }
            if (!dead && from < u.hi && from + 16 > u.lo) {
                const bool whole = from >= u.all_lo && from + 16 <= u.all_hi;
                if (!whole) {
                    // What no row sees counts as 0, and so does a NaN for now: as in kv_attention.cuh.
                    uint8_t *const values = smem + slot * C::STAGE + C::SIDE;
#pragma unroll 1
                    for (int i = lane; i < 16 * KS; i += 32) {
                        const int row = i / KS;
                        uint4 *p = reinterpret_cast<uint4 *>(values + C::at(16 * warp + row, i % KS));
                        const bool seen = from + row >= u.lo && from + row < u.hi, bad = seen && has_nan(*p);
                        if (!seen) *p = make_uint4(0, 0, 0, 0);
                        if (bad) *p = without_nan(*p), *some_nan = 1;
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // (before the next copy into the slot)
                    __syncwarp();
                }
                // S; with few rows in two sums, as one would be a chain of its own latencies
                constexpr int SP = MT == 1 ? 2 : 1;
                float x[MT][2][4], z[MT][2][4];
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[t][n][i] = z[t][n][i] = 0.0f;
#pragma unroll
                for (int k = 0; k < KS; k += 2) {
                    uint32_t a[4];  // 8 and 8 tokens, of two groups of 16 dims
                    ldsm4(sk ^ (k << 4), a);
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int t = 0; t < MT; ++t) {
                            const uint4 q = KEEP ? qf[KEEP ? k + h : 0] : my_q[32 * (KS * t + k + h)];
                            const uint32_t qa[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                            for (int n = 0; n < 2; ++n)
                                mma16816(SP == 2 && h ? z[t][n] : x[t][n], qa, halves(a[h + 2 * n]), halves_hi(a[h + 2 * n]));
                        }
                }
                if constexpr (SP == 2) {
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[0][n][i] += z[0][n][i];
                }
                const float *const scales = sc + SCALES * slot + warp;
                const float ks = scales[0], lv = scales[8], iv = scales[16] * L_FACTOR;
                bool grown = false;
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[t][n][i] = fmaf(x[t][n][i], f[t][i >> 1] * ks, lv);
                if (!whole) {
#pragma unroll
                    for (int t = 0; t < MT; ++t)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int lo = row_lo[16 * t + g + 8 * h], hi = row_hi[16 * t + g + 8 * h];
#pragma unroll
                            for (int n = 0; n < 2; ++n)
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    const int k = 8 * n + 2 * c + i;
                                    float &y = x[t][n][2 * h + i];
                                    if (from + k < lo || from + k >= hi) y = -INFINITY;
                                }
                        }
                }
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float top = fmaxf(fmaxf(x[t][0][2 * h], x[t][0][2 * h + 1]), fmaxf(x[t][1][2 * h], x[t][1][2 * h + 1]));
                        grown |= top > m[t][h] + move;
                    }
                if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
                    for (int t = 0; t < MT; ++t)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float top = fmaxf(fmaxf(x[t][0][2 * h], x[t][0][2 * h + 1]), fmaxf(x[t][1][2 * h], x[t][1][2 * h + 1]));
                            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                            top = top > m[t][h] + move ? top : m[t][h];  // (by this row alone, whatever the others do)
                            const float alpha = ex2(m[t][h] - (top == -INFINITY ? 0.0f : top));
                            m[t][h] = top;
                            l[t][h] *= alpha;
#pragma unroll
                            for (int n = 0; n < DP / 8; ++n) o[t][n][2 * h] *= alpha, o[t][n][2 * h + 1] *= alpha;
                        }
                }
                // P, the operand of the second product
                uint32_t p[MT][4];
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float sub = (m[t][h] == -INFINITY ? 0.0f : m[t][h]) - C::SHIFT;  // (a row that has seen nothing yet: any finite one)
                        float e[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) e[i] = ex2(x[t][i >> 1][2 * h + (i & 1)] - sub);
                        l[t][h] = fmaf((e[0] + e[1]) + (e[2] + e[3]), iv, l[t][h]);
                        p[t][h] = pack2(e[0], e[1]), p[t][2 + h] = pack2(e[2], e[3]);
                    }
                // O: dims 32 d + 16 n + 4 c .. + 3 of the rows, even ones and odd ones
#pragma unroll
                for (int d = 0; d < DP / 32; ++d) {
                    uint32_t a[4];
                    ldsm4_t(sv ^ (d << 5), a);
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        const uint32_t c0 = __byte_perm(a[2 * n], 0, 0x3120), c1 = __byte_perm(a[2 * n + 1], 0, 0x3120);
                        const uint32_t b[2][2] = {{halves(c0), halves(c1)}, {halves_hi(c0), halves_hi(c1)}};
#pragma unroll
                        for (int t = 0; t < MT; ++t)
#pragma unroll
                            for (int i = 0; i < 2; ++i) mma16816(o[t][4 * d + 2 * n + i], p[t], b[i][0], b[i][1]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0 && !dead) mbar_arrive(empty + 8 * slot);
        }

        if (far) {
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int h = 0; h < 2; ++h) l[t][h] = apart[t][h].at(m[t][h]);
        }
        // the warps' maxima and sums, then their O: joined, 16 rows at a time
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                l[t][h] += __shfl_xor_sync(0xffffffffu, l[t][h], 1);
                l[t][h] += __shfl_xor_sync(0xffffffffu, l[t][h], 2);
                const int r = 16 * t + g + 8 * h;
                if (c == 0) warp_m[warp * R + r] = m[t][h], warp_l[warp * R + r] = l[t][h];
            }
        far = named_barrier_or(1, THREADS, far);
        const bool nans = *some_nan != 0;  // (the same for all warps: none is past the next barrier)
        auto out = [&](int r, int64_t &at, int64_t &row) {
            const int i = token_of(P, r0 + r), h = head * P.group + (r0 + r - i * P.group);
            at = (static_cast<int64_t>(s.row0) + i) * P.ldy_t + static_cast<int64_t>(h) * P.ldy_h;
            row = (static_cast<int64_t>(s.row0) + i) * P.heads * P.group + h;
        };
        const bool entire = u.nt == s.tiles;
        // (an entire unit's results, or a part of it: [row][dim] sums relative to the reference, then it and the sum)
        float *const mine = P.part + (static_cast<int64_t>(blockIdx.x) * 2 + (w.tile == 0)) * C::PART;
#pragma unroll
        for (int t = 0; t < MT; ++t) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = 16 * t + g + 8 * h;
                float top = -INFINITY, sum = 0.0f;
#pragma unroll
                for (int k = 0; k < 8; ++k) top = fmaxf(top, warp_m[k * R + r]);
                const float ref = top == -INFINITY ? 0.0f : top, scale = ex2(m[t][h] - ref);
#pragma unroll
                for (int k = 0; k < 8; ++k) sum = fmaf(warp_l[k * R + r], ex2(warp_m[k * R + r] - ref), sum);
                if (far) {  // (as where parts are joined)
                    sum = 0.0f;
#pragma unroll 1
                    for (int k = 0; k < 8; ++k) sum += faded(warp_l[k * R + r], warp_m[k * R + r] - ref);
                }
                if (warp == 0 && c == 0) row_m[r] = top, row_l[r] = sum;
                float *const d = sums + (warp * 16 + g + 8 * h) * C::SUM_ROW + 4 * c;
#pragma unroll
                for (int n = 0; n < DP / 16; ++n)
                    *reinterpret_cast<float4 *>(d + 16 * n) = make_float4(o[t][2 * n][2 * h] * scale, o[t][2 * n + 1][2 * h] * scale,
                                                                          o[t][2 * n][2 * h + 1] * scale, o[t][2 * n + 1][2 * h + 1] * scale);
            }
            named_barrier(1, THREADS);
            for (int i = tid; i < 16 * (DP / 4); i += THREADS) {
                const int rr = i / (DP / 4), r = 16 * t + rr, d = 4 * (i % (DP / 4));
                if (r >= rows) continue;
                float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float4 a = *reinterpret_cast<const float4 *>(sums + (k * 16 + rr) * C::SUM_ROW + d);
                    y.x += a.x, y.y += a.y, y.z += a.z, y.w += a.w;
                }
                const float top = row_m[r], sum = row_l[r];
                if (!entire) {
                    *reinterpret_cast<float4 *>(mine + r * DP + d) = y;
                    if (d == 0) mine[R * DP + r] = top, mine[R * (DP + 1) + r] = sum;
                    continue;
                }
                int64_t at, row;
                out(r, at, row);
                const float inv = sum != 0.0f ? L_FACTOR / sum : 0.0f;
                if (d < P.dim) {
                    store_typed(P.y, at + d, P.y_type, y.x * inv);
                    store_typed(P.y, at + d + 1, P.y_type, y.y * inv);
                    store_typed(P.y, at + d + 2, P.y_type, y.z * inv);
                    store_typed(P.y, at + d + 3, P.y_type, y.w * inv);
                }
                if (P.lse && d == 0) P.lse[row] = sum != 0.0f ? (top + log2f(sum) + 20.0f - C::SHIFT) * LN2 : -INFINITY;
            }
            named_barrier(1, THREADS);
        }
        if (nans) {
            spread_nans(P, w.b, head, start, r0, 0, rows, 0, DP, max(u.from + u.jb * TILE, u.lo), min(u.from + u.je * TILE, u.hi), u.all_lo,
                        u.all_hi, tid, THREADS, [&](int r, int d) {
                            int64_t at, row;
                            out(r, at, row);
                            if (entire) store_typed(P.y, at + d, P.y_type, __uint_as_float(A_NAN));
                            else mine[r * DP + d] = __uint_as_float(A_NAN);
                        });
            named_barrier(1, THREADS);
        }
        if (!entire) {
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

template <int DP, int MT>
cudaError_t launch_one(const AttnParams &p, cudaStream_t st, int num_sms, int dev) {
    using C = Slim<DP, MT>;
    const auto kern = kv_attention_slim_kernel<DP, MT>;
    static OncePerDevice ready;
    const cudaError_t e = ready(dev, [&] {
        cudaError_t r = set_smem_attrs(kern, C::SMEM);
        if (r != cudaSuccess) return r;
        // setmaxnreg draws on what the launch brings
        cudaFuncAttributes fa;
        if ((r = cudaFuncGetAttributes(&fa, kern)) != cudaSuccess) return r;
        return fa.numRegs < REGS ? cudaErrorNotSupported : cudaSuccess;
    });
    if (e != cudaSuccess) return e;
    CUtensorMap tk = {}, tv = {};
    if (!encode_pages(&tk, p.codes[0], p, C::ROW) || !encode_pages(&tv, p.codes[1], p, C::ROW)) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(num_sms));
    cfg.blockDim = dim3(SLIM_THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, tk, tv, p);
}

}  // namespace

cudaError_t launch_slim(const AttnParams &p, int rows, cudaStream_t st, int num_sms, int dev) {
    if (p.dim <= 64) return rows <= 16 ? launch_one<64, 1>(p, st, num_sms, dev) : launch_one<64, 2>(p, st, num_sms, dev);
    return rows <= 16 ? launch_one<128, 1>(p, st, num_sms, dev) : launch_one<128, 2>(p, st, num_sms, dev);
}

}  // namespace kv
}  // namespace qk
