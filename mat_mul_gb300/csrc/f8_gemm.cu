// f8_gemm.cu -- y = W.x with W and x in e4m3 codes, an fp32 scale per
// 128 x 128 block of W and per 128 values of a row of x, over one matrix or
// over groups of rows with a matrix each (experts); optionally the gated pair
// h = silu(Wg.x) * (Wu.x) written back as codes and scales.
//
//   y[r, n] = sum_b  xs[b, r] * Ws[n/128, b] * sum_{k in block b} xq[r, k] W[n, k]
//
// The inner sums run on the fifth-generation tensor cores (tcgen05
// kind::f8f6f4, fp32 accumulation: products of two e4m3 values are exact in
// fp32), one 128-wide block of K at a time into a fresh TMEM buffer; the
// epilogue warps take each finished block out of TMEM and add it, times its
// two scales, to fp32 accumulators in registers.  The scales change from
// block to block and are arbitrary fp32, so they cannot ride inside the MMA.
//
// The weights are the M operand: TMEM lane = weight row n, TMEM column =
// token.  One scale of W covers all 128 lanes of a tile, the number of token
// columns follows the rows there are (16 .. 256 in steps of 16, so a group
// of three rows costs a 16-column MMA), a warp's 32 lanes are 32 consecutive
// n of one row of y, and for the gated pair the 128 lanes of a token are
// exactly one scale block of h.
//
// A tile is 128 weight rows x up to BT tokens.  The grid is one CTA per SM.
// Whole rounds of tiles go round the CTAs; the tiles that would leave the last
// round partly empty (all of them when they are fewer than the CTAs) are cut
// along K so that every CTA has the same number of K blocks.  The CTAs that
// share a tile put their fp32 partial tiles into the workspace, and the last
// one to arrive adds them in K order and stores: no CTA waits for another,
// and the order of the sum does not depend on which one is last.
//
// Warp roles: 0 = copies (TMA, 128-byte swizzle), 1 = MMA issue, 2 = scales,
// 3 = tensor memory; 4..11 = epilogue (warp w: TMEM lanes 32*(w%4), token
// columns of half (w-4)/4).  All waits are bounded.
#include "f8_gemm.cuh"

namespace qk {

namespace {

using namespace f8;

constexpr int BW = 128;
constexpr int THREADS = 384;
constexpr int SC_STAGES = 4;
constexpr int SMEM_MAX = 232448;

template <int BT, bool DUAL>
struct Cfg {
    static constexpr int NA = DUAL ? 2 : 1;            // weight matrices per tile
    // K blocks per step: every wait and hand-over of a step costs the roles a
    // few hundred cycles, about what a 16 KB weight block takes to arrive
    static constexpr int KS = BT <= (DUAL ? 32 : 64) ? 2 : 1;
    static constexpr int XBOX = BT < 64 ? BT : 64;     // rows per token copy
    static constexpr int W_BYTES = BW * BK, X_BYTES = BT * BK;
    static constexpr int BLOCK = NA * W_BYTES + X_BYTES, STAGE = KS * BLOCK;
    static constexpr int SC_FLOATS = BT + 4;           // a K block's scales: of the tokens, of the weights
    static constexpr int SC_BYTES = KS * SC_FLOATS * 4;
    static constexpr int HALF = BT / 2;                // token columns per epilogue warp
    static constexpr int CH = HALF < 16 ? HALF : 16;   // columns per TMEM load
    static constexpr int AMAX_BYTES = DUAL ? 4 * BT * 4 : 0;
    static constexpr int CUM_BYTES = (QMM_F8_MAX_EXPERTS + 4) * 4;
    static constexpr int FIXED = SC_STAGES * SC_BYTES + AMAX_BYTES + CUM_BYTES + 512 + 1024;
    static constexpr int FIT = (SMEM_MAX - FIXED) / STAGE;
    static constexpr int STAGES = FIT > 8 ? 8 : FIT;
    static constexpr int OFF_SC = STAGES * STAGE;
    static constexpr int OFF_AMAX = OFF_SC + SC_STAGES * SC_BYTES;
    static constexpr int OFF_CUM = OFF_AMAX + AMAX_BYTES;
    static constexpr int OFF_BAR = OFF_CUM + CUM_BYTES;
    static constexpr int SMEM = OFF_BAR + 512 + 1024;
    static constexpr int D_COLS = KS * NA * BT;        // one TMEM buffer: a step's sums
    static constexpr int TMEM_COLS = 2 * D_COLS < 32 ? 32 : 2 * D_COLS;
    static constexpr int PART = NA * BT * BW;          // floats of a partial tile
    static_assert(STAGES >= 3 && SMEM <= SMEM_MAX, "shared memory");
    static_assert(TMEM_COLS <= 512, "tensor memory");
    static_assert(8 * (2 * STAGES + 2 * SC_STAGES + 5) + 32 <= 480, "barrier area");
};

struct Params {
    const float *Ws, *W2s, *xs;
    int64_t ld_s;
    const int32_t *offsets;
    int E, R, N, nb, kb;
    int y_type;
    void *y;
    int64_t ldy;
    uint8_t *hq;
    int64_t ld_h;
    float *hs;
    int64_t ld_hs;
    float *part;
    unsigned *count;
    int *status;
    int stop;  // the first CTA issues no copy from this step on (failure test hook)
};

// D[tmem] (+)= A[smem] . B[smem]^T, e4m3 x e4m3 -> fp32
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void store_y(void *y, int type, int64_t i, float v) {
    if (type == QMM_F32) static_cast<float *>(y)[i] = v;
    else if (type == QMM_F16) static_cast<__half *>(y)[i] = __float2half_rn(v);
    else static_cast<__nv_bfloat16 *>(y)[i] = __float2bfloat16_rn(v);
}

template <int BT, bool DUAL>
__global__ void __launch_bounds__(THREADS, 1)
    f8_gemm_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmW2,
                   const __grid_constant__ CUtensorMap tmX, const Params P) {
    using C = Cfg<BT, DUAL>;
    constexpr int NA = C::NA, KS = C::KS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    const uint32_t stage0 = smem_u32(smem);
    const uint32_t bar = smem_u32(smem + C::OFF_BAR);
    const uint32_t full = bar, empty = full + 8 * C::STAGES;
    const uint32_t sc_full = empty + 8 * C::STAGES, sc_empty = sc_full + 8 * SC_STAGES;
    const uint32_t d_full = sc_empty + 8 * SC_STAGES, d_empty = d_full + 16;
    const uint32_t done = d_empty + 16;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_BAR + 480);
    volatile unsigned *arrived = reinterpret_cast<volatile unsigned *>(smem + C::OFF_BAR + 488);
    int *cum = reinterpret_cast<int *>(smem + C::OFF_CUM);

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(full + 8 * s, 1);
            mbar_init(empty + 8 * s, 1);
        }
        for (int s = 0; s < SC_STAGES; ++s) {
            mbar_init(sc_full + 8 * s, 32);
            mbar_init(sc_empty + 8 * s, 8);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(d_full + 8 * s, 1);
            mbar_init(d_empty + 8 * s, 8);
        }
        mbar_init(done, 1);
        fence_mbar_init();
    }
    if (warp == 3) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(C::TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (warp == 0) {
        // only the codes and scales of x come from the launch before this one;
        // the offsets were complete before it started
        f8::count_tiles(cum, P.offsets, P.E, P.R, BT, P.nb, lane, P.status);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    Schedule sch;
    sch.cum = cum;
    sch.offsets = P.offsets;
    sch.E = P.E;
    sch.R = P.R;
    sch.kb = P.kb;
    sch.nb = P.nb;
    sch.G = static_cast<int>(gridDim.x);
    sch.c = static_cast<int>(blockIdx.x);
    sch.step = 0;
    sch.init();
    Piece p;

    if (warp == 0) {
        if (elect_one()) {
            // Copies.  The weights of the first steps are asked for before the
            // launch in front is done (it writes only the codes and scales of x),
            // so that they stream in while x is quantised.
            int stop = NO_STOP;
            if (blockIdx.x == 0 && P.stop != NO_STOP) {  // the failure test hook: at the latest the last step is left out
                Schedule all = sch;
                for (stop = -1; all.next(p);) stop += (p.k1 - p.k0 + KS - 1) / KS;
                stop = min(stop, P.stop);
            }
            int it = 0, early = 0;
            bool ok = true;
            auto weights = [&](const Piece &q, int k, int s) {
                const int kc = min(KS, q.k1 - k), wrow = q.e * P.N + q.nblk * BW;
                const int boxes = (q.ntok + C::XBOX - 1) / C::XBOX;
                const uint32_t st = stage0 + s * C::STAGE, b = full + 8 * s;
                mbar_arrive_expect_tx(b, kc * (NA * C::W_BYTES + boxes * C::XBOX * BK));
                for (int j = 0; j < kc; ++j) {
                    tma_2d(st + j * C::BLOCK, &tmW, (k + j) * BK, wrow, b);
                    if constexpr (DUAL) tma_2d(st + j * C::BLOCK + C::W_BYTES, &tmW2, (k + j) * BK, wrow, b);
                }
            };
            {
                Schedule first = sch;
                while (early < C::STAGES && early < stop && first.next(p))
                    for (int k = p.k0; k < p.k1 && early < C::STAGES && early < stop; k += KS, ++early) weights(p, k, early);
            }
            pdl_wait();
            pdl_trigger();
            while (ok && sch.next(p)) {
                const int boxes = (p.ntok + C::XBOX - 1) / C::XBOX;
                for (int k = p.k0; k < p.k1; k += KS, ++it) {
                    const int s = it % C::STAGES;
                    if (it >= stop ||
                        (it >= C::STAGES && !mbar_spin(empty + 8 * s, ((it / C::STAGES) - 1) & 1, P.status))) {
                        ok = false;
                        break;
                    }
                    if (it >= early) weights(p, k, s);
                    const uint32_t st = stage0 + s * C::STAGE + NA * C::W_BYTES, b = full + 8 * s;
                    const int kc = min(KS, p.k1 - k);
                    for (int j = 0; j < kc; ++j)
                        for (int x = 0; x < boxes; ++x)
                            tma_2d(st + j * C::BLOCK + x * C::XBOX * BK, &tmX, (k + j) * BK, p.row0 + x * C::XBOX, b);
                }
            }
            // no CTA ends with copies in flight
            for (int i = it > C::STAGES ? it - C::STAGES : 0; i < it; ++i)
                mbar_spin(full + 8 * (i % C::STAGES), (i / C::STAGES) & 1, P.status);
        }
    } else if (warp == 1) {
        if (elect_one()) {
            int it = 0;
            bool ok = true;
            while (ok && sch.next(p)) {
                const uint32_t cols = (p.ntok + 15) & ~15;
                const uint32_t idesc = (1u << 4) | ((cols >> 3) << 17) | ((BW >> 4) << 24);
                for (int k = p.k0; k < p.k1; k += KS, ++it) {
                    const int s = it % C::STAGES, d = it & 1;
                    if (!mbar_spin(full + 8 * s, (it / C::STAGES) & 1, P.status) ||
                        (it >= 2 && !mbar_spin(d_empty + 8 * d, ((it >> 1) - 1) & 1, P.status))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
#pragma unroll
                    for (int j = 0; j < KS; ++j) {
                        if (k + j >= p.k1) break;
                        const uint32_t st = stage0 + s * C::STAGE + j * C::BLOCK;
                        const uint64_t b = smem_desc(st + NA * C::W_BYTES);
#pragma unroll
                        for (int m = 0; m < NA; ++m) {
                            const uint64_t a = smem_desc(st + m * C::W_BYTES);
#pragma unroll
                            for (int q = 0; q < BK / 32; ++q)
                                mma_f8(tmem + d * C::D_COLS + (j * NA + m) * BT, a + 2 * q, b + 2 * q, idesc, q ? 1u : 0u);
                        }
                    }
                    mma_commit(empty + 8 * s);
                    mma_commit(d_full + 8 * d);
                }
            }
            mma_commit(done);
        }
    } else if (warp == 2) {
        // Scales of a step, by asynchronous copies straight into shared memory.
        pdl_wait();
        int it = 0;
        bool ok = true;
        while (ok && sch.next(p)) {
            const int64_t ws = (static_cast<int64_t>(p.e) * P.nb + p.nblk) * P.kb;
            const float *w = (DUAL && lane == 1 ? P.W2s : P.Ws) + ws;
            const float *x = P.xs + p.row0;
            for (int k = p.k0; k < p.k1; k += KS, ++it) {
                const int s = it % SC_STAGES;
                if (it >= SC_STAGES)
                    ok = __all_sync(0xffffffffu, mbar_spin(sc_empty + 8 * s, ((it / SC_STAGES) - 1) & 1, P.status));
                if (!ok) break;
                const uint32_t dst = smem_u32(smem + C::OFF_SC) + s * C::SC_BYTES;
                const int kc = min(KS, p.k1 - k);
                for (int j = 0; j < kc; ++j) {
                    for (int t = lane; t < BT; t += 32)
                        copy4(dst + 4 * (j * C::SC_FLOATS + t), x + (k + j) * P.ld_s + min(t, p.ntok - 1));
                    if (lane < NA) copy4(dst + 4 * (j * C::SC_FLOATS + BT + lane), w + k + j);
                }
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(sc_full + 8 * s) : "memory");
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp >= 4) {
        const int quarter = warp & 3, half = (warp - 4) >> 2;
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(32 * quarter) << 16) + half * C::HALF;
        pdl_wait();
        int it = 0;
        bool ok = true;
        while (ok && sch.next(p)) {
            float acc[NA][C::HALF];
#pragma unroll
            for (int m = 0; m < NA; ++m)
#pragma unroll
                for (int i = 0; i < C::HALF; ++i) acc[m][i] = 0.0f;
            const int mine = min(C::HALF, p.ntok - half * C::HALF);  // this warp's token columns (may be <= 0)
            for (int k = p.k0; k < p.k1; k += KS, ++it) {
                const int d = it & 1, s = it % SC_STAGES;
                ok = mbar_spin(sc_full + 8 * s, (it / SC_STAGES) & 1, P.status) &&
                     mbar_spin(d_full + 8 * d, (it >> 1) & 1, P.status);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                const float *sc = reinterpret_cast<const float *>(smem + C::OFF_SC + s * C::SC_BYTES);
                if (mine > 0) {
#pragma unroll
                    for (int j = 0; j < KS; ++j) {
                        if (k + j >= p.k1) break;
#pragma unroll
                        for (int m = 0; m < NA; ++m) {
                            const float w = sc[j * C::SC_FLOATS + BT + m];
#pragma unroll
                            for (int c = 0; c < C::HALF; c += C::CH)
                                if (c < mine) {
                                    uint32_t r[C::CH];
                                    tmem_ld(lane_base + d * C::D_COLS + (j * NA + m) * BT + c, r);
                                    tmem_wait(r);
#pragma unroll
                                    for (int i = 0; i < C::CH; i += 4) {
                                        const float4 f =
                                            *reinterpret_cast<const float4 *>(sc + j * C::SC_FLOATS + half * C::HALF + c + i);
                                        acc[m][c + i] = fmaf(__uint_as_float(r[i]), f.x * w, acc[m][c + i]);
                                        acc[m][c + i + 1] = fmaf(__uint_as_float(r[i + 1]), f.y * w, acc[m][c + i + 1]);
                                        acc[m][c + i + 2] = fmaf(__uint_as_float(r[i + 2]), f.z * w, acc[m][c + i + 2]);
                                        acc[m][c + i + 3] = fmaf(__uint_as_float(r[i + 3]), f.w * w, acc[m][c + i + 3]);
                                    }
                                }
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(d_empty + 8 * d);
                    mbar_arrive(sc_empty + 8 * s);
                }
            }
            // every epilogue warp passes here once per piece, also after a wait
            // that gave up, so that none is left at a barrier alone
            if (named_barrier_or(1, 256, !ok)) break;
            bool store = true;
            if (p.k1 - p.k0 < P.kb) {
                // a part of a cut tile: into the workspace; the last of its
                // CTAs adds the parts in K order
                int c0, c1;
                sch.sharers(p.tile, c0, c1);
                float *mypart = P.part + (static_cast<int64_t>(blockIdx.x) * 2 + (p.k0 == 0)) * C::PART;
#pragma unroll
                for (int m = 0; m < NA; ++m)
#pragma unroll
                    for (int i = 0; i < C::HALF; ++i)
                        if (i < mine)
                            mypart[(m * BT + half * C::HALF + i) * BW + 32 * quarter + lane] = acc[m][i];
                __threadfence();
                named_barrier(1, 256);
                if (threadIdx.x == 128) *arrived = atomicAdd(P.count + c0, 1u);
                named_barrier(1, 256);
                store = *arrived == static_cast<unsigned>(c1 - c0);
                if (store) {
                    if (threadIdx.x == 128) P.count[c0] = 0u;  // zero again for the next launch
                    __threadfence();
#pragma unroll
                    for (int m = 0; m < NA; ++m)
#pragma unroll
                        for (int i = 0; i < C::HALF; ++i) acc[m][i] = 0.0f;
                    // (the parts of a few CTAs at a time, so that their loads overlap)
                    constexpr int U = NA * C::HALF <= 32 ? 32 / (NA * C::HALF) : 1;
                    for (int c = c0; U == 1 && c <= c1; ++c) {
                        const float *q = P.part + (static_cast<int64_t>(c) * 2 + (c == c0)) * C::PART;
#pragma unroll
                        for (int m = 0; m < NA; ++m)
#pragma unroll
                            for (int i = 0; i < C::HALF; ++i)
                                if (i < mine)
                                    acc[m][i] += __ldcg(q + (m * BT + half * C::HALF + i) * BW + 32 * quarter + lane);
                    }
                    for (int c = c0; U > 1 && c <= c1; c += U) {
                        float v[U][NA][C::HALF];
#pragma unroll
                        for (int u = 0; u < U; ++u) {
                            const float *q = P.part + (static_cast<int64_t>(c + u) * 2 + (c + u == c0)) * C::PART;
#pragma unroll
                            for (int m = 0; m < NA; ++m)
#pragma unroll
                                for (int i = 0; i < C::HALF; ++i)
                                    v[u][m][i] = c + u <= c1 && i < mine
                                                     ? __ldcg(q + (m * BT + half * C::HALF + i) * BW + 32 * quarter + lane)
                                                     : 0.0f;
                        }
#pragma unroll
                        for (int u = 0; u < U; ++u)
#pragma unroll
                            for (int m = 0; m < NA; ++m)
#pragma unroll
                                for (int i = 0; i < C::HALF; ++i) acc[m][i] += v[u][m][i];
                    }
                }
            }
            if (!store) continue;
            const int n = p.nblk * BW + 32 * quarter + lane;
            const int64_t row = p.row0 + half * C::HALF;
            if constexpr (!DUAL) {
                if (n < P.N) {
#pragma unroll
                    for (int i = 0; i < C::HALF; ++i)
                        if (i < mine) store_y(P.y, P.y_type, (row + i) * P.ldy + n, acc[0][i]);
                }
            } else {
                // h = silu(g) * u, its largest |h| over the tile's 128 rows n
                // (one scale block of h), then its codes
                uint32_t *amax = reinterpret_cast<uint32_t *>(smem + C::OFF_AMAX) + half * C::HALF;
#pragma unroll
                for (int i = 0; i < C::HALF; ++i)
                    if (i < mine) {
                        const float g = acc[0][i];
                        const float h = n < P.N ? silu(g) * acc[1][i] : 0.0f;
                        acc[0][i] = h;
                        const uint32_t a = __reduce_max_sync(0xffffffffu, __float_as_uint(h) & 0x7fffffffu);
                        if (lane == 0) amax[quarter * BT + i] = a;
                    }
                named_barrier(2 + half, 128);
#pragma unroll
                for (int i = 0; i < C::HALF; ++i)
                    if (i < mine) {
                        const uint32_t a = max(max(amax[i], amax[BT + i]), max(amax[2 * BT + i], amax[3 * BT + i]));
                        float s = __fdiv_rn(__uint_as_float(a), 448.0f);
                        s = s < 1.17549435e-38f ? 1.17549435e-38f : s;
                        if (n < P.N)
                            P.hq[(row + i) * P.ld_h + n] =
                                __nv_cvt_float_to_fp8(acc[0][i] * __fdiv_rn(1.0f, s), __NV_SATFINITE, __NV_E4M3);
                        if (quarter == 0 && lane == 0) P.hs[p.nblk * P.ld_hs + row + i] = s;
                    }
                named_barrier(2 + half, 128);  // amax may be overwritten
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 3) {
        mbar_spin(done, 0, P.status);  // every MMA has completed
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::TMEM_COLS)
                     : "memory");
    }
}

template <int BT, bool DUAL>
cudaError_t launch_bt(const F8Gemm &g, cudaStream_t st, int num_sms) {
    using C = Cfg<BT, DUAL>;
    CUtensorMap tw = {}, tw2 = {}, tx = {};
    if (!encode_rows(&tw, g.W, g.E * g.N, g.K, g.K, BW) || (DUAL && !encode_rows(&tw2, g.W2, g.E * g.N, g.K, g.K, BW)) ||
        !encode_rows(&tx, g.xq, g.R, g.K, g.ld_q, C::XBOX))
        return cudaErrorInvalidValue;
    Params p = {};
    p.Ws = g.Ws;
    p.W2s = g.W2s;
    p.xs = g.xs;
    p.ld_s = g.ld_s;
    p.offsets = g.offsets;
    p.E = g.E;
    p.R = static_cast<int>(g.R);
    p.N = static_cast<int>(g.N);
    p.nb = static_cast<int>(f8_blocks(g.N));
    p.kb = static_cast<int>(f8_blocks(g.K));
    p.y_type = g.y_type;
    p.y = g.y;
    p.ldy = g.ldy;
    p.hq = g.hq;
    p.ld_h = g.ld_h;
    p.hs = g.hs;
    p.ld_hs = g.ld_hs;
    p.part = g.part;
    p.count = g.count;
    p.status = g.status;
    p.stop = inject_stop_stage();
    static OncePerDevice ready;
    const cudaError_t e = ready(g.dev, [] { return set_smem_attrs(f8_gemm_kernel<BT, DUAL>, C::SMEM); });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(num_sms));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, f8_gemm_kernel<BT, DUAL>, tw, tw2, tx, p);
}

// Tokens per tile: the mean rows of a group, rounded up to a tile width.
int tile_tokens(int64_t R, int E) {
    const int64_t mean = (R + E - 1) / E;
    int bt = 16;
    while (bt < mean && bt < 128) bt *= 2;
    return bt;
}

// Which kernel: 0 this one, 1 f8_wide.cu on single CTAs, 2 on pairs.
int path_of(int64_t R, int E) {
    const int64_t mean = (R + E - 1) / E;
    if (mean <= 128) return 0;
    return E == 1 || mean > 1024 ? 2 : 1;
}

template <bool DUAL>
cudaError_t launch_any(const F8Gemm &g, cudaStream_t st, int num_sms) {
    if (const int w = path_of(g.R, g.E)) return launch_f8_wide(g, w == 2, st, num_sms);
    switch (tile_tokens(g.R, g.E)) {
    case 16: return launch_bt<16, DUAL>(g, st, num_sms);
    case 32: return launch_bt<32, DUAL>(g, st, num_sms);
    case 64: return launch_bt<64, DUAL>(g, st, num_sms);
    default: return launch_bt<128, DUAL>(g, st, num_sms);
    }
}

}  // namespace

size_t f8_part_bytes(int64_t R, int E, bool dual, int num_sms) {
    if (path_of(R, E)) return f8_wide_part_bytes(num_sms);
    return static_cast<size_t>(num_sms) * 2 * (dual ? 2 : 1) * tile_tokens(R, E) * BW * sizeof(float);
}

bool f8_available() { return tensor_map_encoder() != nullptr; }

cudaError_t launch_f8_gemm(const F8Gemm &g, cudaStream_t st, int num_sms) {
    return g.W2 ? launch_any<true>(g, st, num_sms) : launch_any<false>(g, st, num_sms);
}

}  // namespace qk
