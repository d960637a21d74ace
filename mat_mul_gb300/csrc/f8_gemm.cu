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
// This kernel is for groups of few rows (f8_wide.cu takes the others), where the
// reading of the weights is what there is to do.  The weights are the M operand:
// TMEM lane = weight row n, TMEM column = token.  One scale of W covers all 128
// lanes of a tile, the number of token columns follows the rows there are (16 ..
// 64 in steps of 16, so a group of three rows costs a 16-column MMA), a warp's 32
// lanes are 32 consecutive n of one row of y, and for the gated pair the 128
// lanes of a token are exactly one scale block of h.
//
// A tile is 128 weight rows x up to BT tokens.  The grid is one CTA per SM.
// Whole rounds of tiles go round the CTAs; where the last round would leave too
// many CTAs idle for too long its tiles are cut along K (Schedule::plan).  The CTAs that
// share a tile put their fp32 partial tiles into the workspace, and the last
// one to arrive adds them in K order and stores: no CTA waits for another,
// and the order of the sum does not depend on which one is last.
//
// Measured out of HBM (bf16, a row of calls on different matrices): 1 x 4096 x
// 14336 14.8 us (4.0 TB/s of the 59 MB, 0.59 of the measured copy rate), 1 x 5120
// x 17408 19.0 us (4.7 TB/s), 64 rows of 64 experts of 2048 x 1536 (41 of them in
// use) 27.3 us (4.7 TB/s): about 6 us, the launches and the start and end of the
// pipeline, plus the weights at 6.8 TB/s.  What bounds it below about 100 MB is
// therefore latency: the launch, the first weights, then per step the hand-over
// from the copies to the MMA to the epilogue, and the sum over the CTAs of a tile.
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
constexpr int LEAST = 4;  // K blocks of cut tiles per CTA (13 x 5120 x 1024: with two 10.1 us, four 9.3, sixteen 12.7)
constexpr int FUSE_BLOCKS = 8;   // most K blocks per CTA with FUSE
constexpr int FUSE_WARPS = 10, FUSE_ITEMS = 8;  // warps 2 .. 11 quantise, eight (block, row) items each
constexpr int SMEM_MAX = 232448;

template <int BT, bool DUAL, bool FUSE>
struct Cfg {
    static constexpr int NA = DUAL ? 2 : 1;            // weight matrices per tile
    // K blocks per step: every wait and hand-over of a step costs the roles a
    // few hundred cycles, about what a 16 KB weight block takes to arrive (16 x
    // 4096 x 14336: two blocks per step 15.4 us, four 14.3)
    static constexpr int KS = BT == 16 && !DUAL && !FUSE ? 4 : BT <= (DUAL ? 32 : 64) ? 2 : 1;
    static constexpr int XBOX = BT < 64 ? BT : 64;     // rows per token copy
    static constexpr int W_BYTES = BW * BK, X_BYTES = BT * BK;
    static constexpr int BLOCK = NA * W_BYTES + (FUSE ? 0 : X_BYTES), STAGE = KS * BLOCK;
    static constexpr int SC_FLOATS = BT + 4;           // a K block's scales: of the tokens, of the weights
    static constexpr int SC_BYTES = KS * SC_FLOATS * 4;
    static constexpr int HALF = BT / 2;                // token columns per epilogue warp
    static constexpr int CH = HALF < 16 ? HALF : 16;   // columns per TMEM load
    static constexpr int AMAX_BYTES = DUAL ? 4 * BT * 4 : 0;
    static constexpr int CUM_BYTES = (QMM_F8_MAX_EXPERTS + 4) * 4;
    // FUSE: the codes and the scales of every K block the CTA needs
    static constexpr int OWN_X = FUSE ? FUSE_BLOCKS * X_BYTES : 0, OWN_SC = FUSE ? FUSE_BLOCKS * SC_FLOATS * 4 : 0;
    static constexpr int FIXED = OWN_X + OWN_SC + SC_STAGES * SC_BYTES + AMAX_BYTES + CUM_BYTES + 512 + 1024;
    static constexpr int FIT = (SMEM_MAX - FIXED) / STAGE;
    static constexpr int STAGES = FIT > 8 ? 8 : FIT;
    static constexpr int OFF_X = STAGES * STAGE, OFF_XS = OFF_X + OWN_X;
    static constexpr int OFF_SC = OFF_XS + OWN_SC;
    static constexpr int OFF_AMAX = OFF_SC + SC_STAGES * SC_BYTES;
    static constexpr int OFF_CUM = OFF_AMAX + AMAX_BYTES;
    static constexpr int OFF_BAR = OFF_CUM + CUM_BYTES;
    static constexpr int SMEM = OFF_BAR + 512 + 1024;
    static constexpr int D_COLS = KS * NA * BT;        // one TMEM buffer: a step's sums
    static constexpr int TMEM_COLS = 2 * D_COLS < 32 ? 32 : 2 * D_COLS;
    static constexpr int PART = NA * BT * BW;          // floats of a partial tile
    static_assert(STAGES >= 3 && SMEM <= SMEM_MAX, "shared memory");
    static_assert(TMEM_COLS <= 512, "tensor memory");
    static_assert(8 * (2 * STAGES + 2 * SC_STAGES + 6) <= 480, "barrier area");
    static_assert(!FUSE || (BT == 16 && !DUAL), "FUSE: one tile of tokens, one matrix");
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
    const void *x;  // with FUSE
    int x_type, x_vec, K;
    int64_t ldx;
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

// Four values of x from element c of row r (zeros past K).
__device__ __forceinline__ void load_x4(const Params &P, int r, int c, float (&v)[4]) {
    v[0] = v[1] = v[2] = v[3] = 0.0f;
    if (c >= P.K) return;  // (K is a multiple of 16)
    const int64_t at = r * P.ldx + c;
    if (P.x_type == QMM_F32) {
        const float *x = static_cast<const float *>(P.x) + at;
        if (P.x_vec) {
            const float4 a = *reinterpret_cast<const float4 *>(x);
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = x[i];
        }
        return;
    }
    const uint16_t *x = static_cast<const uint16_t *>(P.x) + at;
    uint32_t a, b;
    if (P.x_vec) {
        const uint2 u = *reinterpret_cast<const uint2 *>(x);
        a = u.x, b = u.y;
    } else {
        a = x[0] | static_cast<uint32_t>(x[1]) << 16;
        b = x[2] | static_cast<uint32_t>(x[3]) << 16;
    }
    if (P.x_type == QMM_F16) {
        const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&a));
        const float2 q = __half22float2(*reinterpret_cast<const __half2 *>(&b));
        v[0] = p.x, v[1] = p.y, v[2] = q.x, v[3] = q.y;
    } else {
        v[0] = __uint_as_float(a << 16), v[1] = __uint_as_float(a & 0xffff0000u);
        v[2] = __uint_as_float(b << 16), v[3] = __uint_as_float(b & 0xffff0000u);
    }
}

// FUSE: the codes of this CTA's K blocks, block b (in the order of its pieces)
// to codes + b * 2048 in the swizzled rows the MMA reads, its scales to
// sc + b * pitch (rows, then the scale of W).  Each warp takes up to eight
// (block, row) items, all of them in flight at once; the same arithmetic as
// f8_quantize.cu, so the codes are the same.
__device__ __forceinline__ void quantise_own(const Params &P, const Schedule &s, uint8_t *codes, float *sc, int pitch,
                                             int warp, int lane) {
    const int cut = s.u1 - s.u;
    const int blocks = cut + (s.whole > s.c ? (s.whole - 1 - s.c) / s.G + 1 : 0) * s.kb;
    const int items = blocks * P.R, i0 = warp * FUSE_ITEMS;  // (at most FUSE_WARPS * FUSE_ITEMS: see f8_fuses)
    auto block_k = [&](int b) { return b < cut ? (s.u + b) % s.kb : (b - cut) % s.kb; };
    // lane g: block and row of item g (the divisions once per item)
    const int i = min(i0 + lane, items - 1), block = i / P.R, row = i - block * P.R, kblk = block_k(block);
    float v[FUSE_ITEMS][4];
#pragma unroll
    for (int g = 0; g < FUSE_ITEMS; ++g) {
        const int r = __shfl_sync(0xffffffffu, row, g), k = __shfl_sync(0xffffffffu, kblk, g);
        if (i0 + g < items) load_x4(P, r, k * BK + 4 * lane, v[g]);
    }
    for (int b = warp * 32 + lane; b < blocks; b += FUSE_WARPS * 32) {
        const int tile = b < cut ? s.whole + (s.u + b) / s.kb : s.c + (b - cut) / s.kb * s.G;
        sc[b * pitch + 16] = __ldg(P.Ws + static_cast<int64_t>(tile) * s.kb + block_k(b));  // (one tile of tokens)
    }
    uint32_t mine = 0;  // lane g: the largest |x| of item g
#pragma unroll
    for (int g = 0; g < FUSE_ITEMS; ++g) {
        if (i0 + g >= items) break;
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) m = max(m, __float_as_uint(v[g][j]) & 0x7fffffffu);
        m = __reduce_max_sync(0xffffffffu, m);
        if (lane == g) mine = m;
    }
    float scale = __fdiv_rn(__uint_as_float(mine), 448.0f);
    scale = scale < 1.17549435e-38f ? 1.17549435e-38f : scale;
    const float inv_mine = __fdiv_rn(1.0f, scale);
    if (lane < FUSE_ITEMS && i0 + lane < items) sc[block * pitch + row] = scale;
#pragma unroll
    for (int g = 0; g < FUSE_ITEMS; ++g) {
        if (i0 + g >= items) break;
        const float inv = __shfl_sync(0xffffffffu, inv_mine, g);
        const int b = __shfl_sync(0xffffffffu, block, g), t = __shfl_sync(0xffffffffu, row, g);
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[g][0] * inv, v[g][1] * inv), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[g][2] * inv, v[g][3] * inv), __NV_SATFINITE, __NV_E4M3);
        *reinterpret_cast<uint32_t *>(codes + b * (16 * BK) + t * BK + ((4 * lane) ^ ((t & 7) << 4))) = lo | hi << 16;
    }
    // the MMA reads shared memory through the asynchronous proxy
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// FUSE (few rows of a small matrix): the kernel quantises x itself, each CTA the K
// blocks it needs: one launch instead of two, which is what counts where the
// host's launches take longer than the GPU's work (13 x 5120 x 1024 10.4 instead
// of 14.5 us a call; on the GPU alone 10.1 against 9.1; a call takes 10 to 15 us,
// depending on the host).  Not where the weights
// take longer than the quantiser's launch, ahead of which they are asked for (1 x
// 4096 x 14336 out of HBM 18.2 against 14.6), and only where every warp's items
// are loaded at once (16 x 4096 x 14336 in five turns took 26 against 14).
template <int BT, bool DUAL, bool FUSE>
__global__ void __launch_bounds__(THREADS, 1)
    f8_gemm_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmW2,
                   const __grid_constant__ CUtensorMap tmX, const Params P) {
    using C = Cfg<BT, DUAL, FUSE>;
    constexpr int NA = C::NA, KS = C::KS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    const uint32_t stage0 = smem_u32(smem);
    const uint32_t bar = smem_u32(smem + C::OFF_BAR);
    const uint32_t full = bar, empty = full + 8 * C::STAGES;
    const uint32_t sc_full = empty + 8 * C::STAGES, sc_empty = sc_full + 8 * SC_STAGES;
    const uint32_t d_full = sc_empty + 8 * SC_STAGES, d_empty = d_full + 16;
    const uint32_t done = d_empty + 16, x_ready = done + 8;
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
        mbar_init(x_ready, FUSE_WARPS);
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
    sch.least = LEAST;
    sch.init();
    Piece p;

    if (warp == 0) {
        if (elect_one()) {
            // Copies.  The launch in front is the quantiser, which writes only the
            // codes and scales of x, so the weights of the first steps are asked
            // for before it is done.  With FUSE it may be any launch: until it is
            // done the weights are brought as far as L2, which is safe whatever
            // it writes.
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
                mbar_arrive_expect_tx(b, kc * (NA * C::W_BYTES + (FUSE ? 0 : boxes * C::XBOX * BK)));
                for (int j = 0; j < kc; ++j) {
                    tma_2d(st + j * C::BLOCK, &tmW, (k + j) * BK, wrow, b);
                    if constexpr (DUAL) tma_2d(st + j * C::BLOCK + C::W_BYTES, &tmW2, (k + j) * BK, wrow, b);
                }
            };
            if constexpr (FUSE) {
                Schedule first = sch;
                while (first.next(p))
                    for (int k = p.k0; k < p.k1; ++k) prefetch_2d(&tmW, k * BK, p.nblk * BW);
            } else {
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
                    if constexpr (FUSE) continue;
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
            int it = 0, blk = 0;
            bool ok = !FUSE || mbar_spin(x_ready, 0, P.status);
            while (ok && sch.next(p)) {
                const uint32_t cols = (p.ntok + 15) & ~15;
                const uint32_t idesc = (1u << 4) | ((cols >> 3) << 17) | ((BW >> 4) << 24);
                for (int k = p.k0; k < p.k1; blk += min(KS, p.k1 - k), k += KS, ++it) {
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
                        const uint64_t b =
                            smem_desc(FUSE ? stage0 + C::OFF_X + (blk + j) * C::X_BYTES : st + NA * C::W_BYTES);
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
    } else if (!FUSE && warp == 2) {
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
    } else if (FUSE || warp >= 4) {
        const int quarter = warp & 3, half = (warp - 4) >> 2;
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(32 * quarter) << 16) + half * C::HALF;
        pdl_wait();
        if constexpr (FUSE) {
            quantise_own(P, sch, smem + C::OFF_X, reinterpret_cast<float *>(smem + C::OFF_XS), C::SC_FLOATS, warp - 2, lane);
            __syncwarp();
            if (lane == 0) mbar_arrive(x_ready);
        }
        int it = 0, blk = 0;
        bool ok = true;
        if constexpr (FUSE) ok = __all_sync(0xffffffffu, mbar_spin(x_ready, 0, P.status));
        while (warp >= 4 && sch.next(p)) {  // (with FUSE warps 2 and 3 only quantise)
            float acc[NA][C::HALF];
#pragma unroll
            for (int m = 0; m < NA; ++m)
#pragma unroll
                for (int i = 0; i < C::HALF; ++i) acc[m][i] = 0.0f;
            const int mine = min(C::HALF, p.ntok - half * C::HALF);  // this warp's token columns (may be <= 0)
            for (int k = p.k0; ok && k < p.k1; blk += min(KS, p.k1 - k), k += KS, ++it) {
                const int d = it & 1, s = it % SC_STAGES;
                ok = (FUSE || mbar_spin(sc_full + 8 * s, (it / SC_STAGES) & 1, P.status)) &&
                     mbar_spin(d_full + 8 * d, (it >> 1) & 1, P.status);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                const float *sc = reinterpret_cast<const float *>(smem + (FUSE ? C::OFF_XS + blk * C::SC_FLOATS * 4
                                                                               : C::OFF_SC + s * C::SC_BYTES));
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
                    if (!FUSE) mbar_arrive(sc_empty + 8 * s);
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
                    constexpr int U = NA * C::HALF <= 64 ? 64 / (NA * C::HALF) : 1;
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

template <int BT, bool DUAL, bool FUSE = false>
cudaError_t launch_bt(const F8Gemm &g, cudaStream_t st, int num_sms) {
    using C = Cfg<BT, DUAL, FUSE>;
    CUtensorMap tw = {}, tw2 = {}, tx = {};
    if (!encode_rows(&tw, g.W, g.E * g.N, g.K, g.K, BW) || (DUAL && !encode_rows(&tw2, g.W2, g.E * g.N, g.K, g.K, BW)) ||
        (!FUSE && !encode_rows(&tx, g.xq, g.R, g.K, g.ld_q, C::XBOX)))
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
    if (FUSE) {
        p.x = g.x;
        p.x_type = g.x_type;
        p.ldx = g.ldx;
        p.K = static_cast<int>(g.K);
        p.x_vec = g.ldx % 4 == 0 && reinterpret_cast<uintptr_t>(g.x) % (4 * f8_size(g.x_type)) == 0;
    }
    p.stop = inject_stop_stage();
    static OncePerDevice ready;
    const cudaError_t e = ready(g.dev, [] { return set_smem_attrs(f8_gemm_kernel<BT, DUAL, FUSE>, C::SMEM); });
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
    return cudaLaunchKernelEx(&cfg, f8_gemm_kernel<BT, DUAL, FUSE>, tw, tw2, tx, p);
}

// Tokens per tile: the mean rows of a group, rounded up to a tile width.
int tile_tokens(int64_t R, int E) {
    const int64_t mean = (R + E - 1) / E;
    int bt = 16;
    while (bt < mean && bt < 64) bt *= 2;
    return bt;
}

// Which kernel: 0 this one, 1 f8_wide.cu on single CTAs, 2 on pairs.  Measured
// (bf16, us; this, single, pair):
//   one matrix of 5120 x 5120: 64 rows 15 22 20, 128 rows 19 23 21, 192 rows 20 21 21,
//     256 rows 27 21 21, 1024 rows 77 39 38
//   of 14336 x 4096: 64 rows 17 21 20, 96 rows 26 20 20, 1024 rows 146 55 52
//   32 experts of 2816 x 2048 (mean rows): 8 22 26 31, 16 32 29 38, 32 43 38 41,
//     128 92 49 60; 4 experts, 2048: 146 59 64
//   32 expert layers of 2048 x 1408: 8 41 49 59, 16 55 58 75, 32 75 67 78, 128 185 92 110
// So this one for as many rows of one matrix as its tiles fit the GPU once (at
// least 64), else pairs; for row groups single CTAs from a mean of 25 rows, whose
// ragged ends a pair's 256 rows would waste.  The mean is over all experts, used
// or not, since the group sizes are on the device.  A few crowded experts among
// idle ones then run here, one tile per 16 of their rows, which costs no more as
// long as the tiles fit the GPU: of 64 experts of 1536 x 2048 one with 64 / 200 / 512 / 1000
// rows and the others empty 10.8 / 12.8 / 16.6 / 24.2 us, that expert alone (single
// CTAs) 16.7 / 16.9 / 18.6 / 18.8.
int path_of(int64_t R, int E, int64_t N, bool grouped, int num_sms) {
    if (grouped) return (R + E - 1) / E <= 24 ? 0 : 1;
    return R <= 64 || (R <= 192 && (R + 63) / 64 * f8_blocks(N) <= num_sms) ? 0 : 2;
}

template <bool DUAL>
cudaError_t launch_any(const F8Gemm &g, cudaStream_t st, int num_sms) {
    if constexpr (!DUAL)
        if (!g.xq) return launch_bt<16, false, true>(g, st, num_sms);
    if (const int w = path_of(g.R, g.E, g.N, g.offsets != nullptr, num_sms)) {
        // (not supported: a build of that kernel with too few registers; its partial tiles take more memory than here)
        const cudaError_t e = launch_f8_wide(g, w, st, num_sms);
        if (e != cudaErrorNotSupported) return e;
    }
    const int bt = tile_tokens(g.R, g.E);
    if (bt == 16) return launch_bt<16, DUAL>(g, st, num_sms);
    if constexpr (!DUAL)
        if (bt == 64) return launch_bt<64, false>(g, st, num_sms);
    return launch_bt<32, DUAL>(g, st, num_sms);  // (the gated pair always has row groups, of 24 in the mean at most)
}

}  // namespace

size_t f8_part_bytes(int64_t R, int E, int64_t N, bool dual, bool grouped, int num_sms) {
    if (path_of(R, E, N, grouped, num_sms)) return f8_wide_part_bytes(num_sms);
    return static_cast<size_t>(num_sms) * 2 * (dual ? 2 : 1) * tile_tokens(R, E) * BW * sizeof(float);
}

bool f8_fuses(int64_t R, int64_t N, int64_t K, int num_sms) {
    if (R > 16 || R < 1) return false;
    // the K blocks of the CTA that has most (see Schedule)
    const int tiles = static_cast<int>(f8_blocks(N)), kb = static_cast<int>(f8_blocks(K));
    int whole, units, sharing;
    Schedule::plan(tiles, kb, num_sms, LEAST, whole, units, sharing);
    const int64_t blocks = static_cast<int64_t>((whole + num_sms - 1) / num_sms) * kb +
                           (sharing ? (units + sharing - 1) / sharing : 0);
    return blocks <= FUSE_BLOCKS && blocks * R <= FUSE_WARPS * FUSE_ITEMS;
}

bool f8_available() { return tensor_map_encoder() != nullptr; }

cudaError_t launch_f8_gemm(const F8Gemm &g, cudaStream_t st, int num_sms) {
    return g.W2 ? launch_any<true>(g, st, num_sms) : launch_any<false>(g, st, num_sms);
}

}  // namespace qk
