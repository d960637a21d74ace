// f8_wide.cu -- the block-scaled 8-bit-float product for groups of many rows:
// the same sums as f8_gemm.cu with the operands' roles exchanged.
//
// Here the tokens are the M operand (TMEM lanes) and 256 weight rows the
// columns, 256 rows of one matrix or 128 of gate and 128 of up.  A thread of
// the epilogue owns one token, and its columns lie in one scale block of W (of
// each matrix, for the gated pair): the factor xs * Ws of a K block is a scalar
// per thread and the block goes from TMEM into fp32 registers at one packed fma
// per two values, while in f8_gemm.cu every column has its own factor in shared
// memory, which the operands of the MMA need for themselves (4096 x 5120 x 17408:
// 776 us there with 256 token columns, 280 to 305 here).
//
// With CG = 2 a pair of CTAs works on 256 tokens x 256 columns with one
// cta_group::2 MMA: each loads its own 128 tokens and half of the weight rows,
// so the copies of W are halved.
//
// What bounds it: a K block takes about 800 cycles, of which the tensor pipe is
// busy 512, about 60 %.  The two TMEM buffers alone would allow a block in about 600
// (a buffer's round is the MMA, its commit, the epilogue's reading of it, about 300
// cycles for 128 columns per warp, and the hand-back).  The thread that issues the
// MMAs takes longer: about 410 cycles for four MMAs and two commits, and 100 to 200
// for each of its two waits, also when the barrier is complete.  That adds up to
// the 800; which part could run beside which was not tried.  Stores of a finished
// tile are another 6 %.
//
// Warp roles: 0 = copies, 1 = MMA issue (of the pair's first CTA), 2 = scales,
// 3 = schedule (and tensor memory), then the epilogue (warp w: TMEM lanes
// 32*(w%4), columns of part (w-4)/4).  Schedule of the tiles, cut tiles and
// bounded waits as in f8_gemm.cu.
#include "f8_gemm.cuh"

namespace qk {

namespace {

using namespace f8;

constexpr int TOK = 128;   // tokens per CTA
constexpr int COLS = 256;  // TMEM columns of a buffer
constexpr int LEAST = 4;   // K blocks of cut tiles per CTA
constexpr int PIECES = 4;  // pieces the scheduling warp is ahead
constexpr int BATCH = 4, SC_RING = 3, SC_FLOATS = TOK + 4;  // scales in shared memory
constexpr int PART = TOK * COLS;              // floats of a partial tile of one CTA
constexpr long long DRAIN_CYCLES = 1 << 21;   // about a millisecond

template <int CG, bool DUAL>
struct Wide {
    static_assert(CG == 1 || !DUAL, "the gated pair has row groups, whose ragged ends the 256 rows of CTA pairs would waste");
    // Epilogue warps per TMEM lane quarter (each has its share of the columns)
    // and the registers they get.  Two warps of 128 accumulators per thread
    // measured faster than four of 64 for one matrix (8192 rows of 40 experts 95
    // against 103 us), slower for the gated pair, whose rounding needs more
    // registers beside them (4093 tokens, 32 experts: 327 against 304 us).  (Figures
    // of an earlier state: 81 and 235 us now.)
    static constexpr int PARTS = DUAL ? 4 : 2;
    static constexpr int EPI = 4 * PARTS, EPI_THREADS = 32 * EPI, THREADS = 128 + EPI_THREADS;
    static constexpr int OWN = COLS / PARTS;  // accumulators per thread
    // registers per thread at launch, and after the split between the first
    // four warps and the epilogue
    static constexpr int REGS = DUAL ? 96 : 168;
    static constexpr int REGS_LOW = DUAL ? 32 : 56, REGS_HIGH = DUAL ? 112 : 224;
    static_assert(128 * REGS_LOW + EPI_THREADS * REGS_HIGH <= THREADS * REGS, "register split");
    static constexpr int CHUNKS = DUAL ? 2 : 4;              // 16-byte chunks of a row that go to memory together
    static constexpr int ROWS_BYTES = 32 * 16 * CHUNKS;      // a warp's rows on their way to memory
    static constexpr int A_BYTES = TOK * BK, B_ROWS = COLS / CG, B_BYTES = B_ROWS * BK;
    static constexpr int STAGE = A_BYTES + B_BYTES;
    static constexpr int STAGES = CG == 2 ? 6 : 4;
    static constexpr int OFF_SC = STAGES * STAGE;  // SC_RING batches of BATCH K blocks: xs of the tokens, two of W
    static constexpr int OFF_AMAX = OFF_SC + SC_RING * BATCH * SC_FLOATS * 4;
    static constexpr int OFF_CUM = OFF_AMAX + PARTS * TOK * 4;
    static constexpr int OFF_PIECES = OFF_CUM + (QMM_F8_MAX_EXPERTS + 4) * 4;
    static constexpr int OFF_ROWS = OFF_PIECES + PIECES * 48;
    static constexpr int OFF_BAR = OFF_ROWS + EPI * ROWS_BYTES;
    static constexpr int SMEM = OFF_BAR + 512 + 1024;
    static_assert(SMEM <= 232448, "shared memory");
};

struct Params {
    const float *Ws, *W2s, *xs;
    int64_t ld_s;
    const int32_t *offsets;
    int E, R, N, nb, tiles_n, kb;
    int y_type, y_vec;
    void *y;
    int64_t ldy;
    uint8_t *hq;
    int64_t ld_h;
    float *hs;
    int64_t ld_hs;
    float *part;
    unsigned *count;
    int *status;
    int stop;
};

template <int CG>
__device__ __forceinline__ void mma_wide(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    if constexpr (CG == 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc)
            : "memory");
}

// Arrive on `bar` (same offset in every CTA of the group) once all MMAs
// issued so far are complete.
template <int CG>
__device__ __forceinline__ void commit(uint32_t bar) {
    if constexpr (CG == 1)
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                     : "memory");
    else
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                bar),
            "h"(static_cast<uint16_t>(3))
            : "memory");
}

// Copy into this CTA's shared memory that completes on `bar`, an address in
// the shared memory of the pair's first CTA.
__device__ __forceinline__ void tma_2d_pair(uint32_t dst, const CUtensorMap *map, int c0, int c1, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// The address in CTA `rank` of the cluster of this CTA's shared address a.
__device__ __forceinline__ uint32_t map_rank(uint32_t a, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    return r;
}
__device__ __forceinline__ void arrive_cluster(uint32_t a) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(a) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// acc[0..1] += (a, b) * (s, s)
__device__ __forceinline__ void fma2(float &x, float &y, uint32_t a, uint32_t b, float s) {
    asm("{\n\t.reg .b64 p, q, r;\n\t"
        "mov.b64 p, {%2, %3};\n\t"
        "mov.b64 q, {%4, %4};\n\t"
        "mov.b64 r, {%0, %1};\n\t"
        "fma.rn.f32x2 r, p, q, r;\n\t"
        "mov.b64 {%0, %1}, r;\n\t}"
        : "+f"(x), "+f"(y)
        : "r"(a), "r"(b), "f"(s));
}

// CHUNKS * 16 bytes of each of the warp's 32 rows (lane = row) to memory:
// through shared memory, so that a store instruction writes whole 64-byte
// pieces of eight rows instead of 16 bytes of 32 (the 4096 x 5120 x 17408
// product: 60 us less).  A row's chunks are permuted so that both accesses
// are free of bank conflicts.  put(row, chunk, data) stores.
template <int CHUNKS, class F>
__device__ __forceinline__ void rows_out(uint8_t *buf, int lane, const uint4 (&w)[CHUNKS], F put) {
    constexpr int PER = 32 / CHUNKS, SH = CHUNKS == 4 ? 1 : 2;  // rows per load, rows that share a permutation
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c)
        *reinterpret_cast<uint4 *>(buf + 16 * (CHUNKS * lane + (c ^ ((lane >> SH) & (CHUNKS - 1))))) = w[c];
    __syncwarp();
    uint4 v[CHUNKS];
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
        const int r = PER * i + lane / CHUNKS, c = lane % CHUNKS;
        v[i] = *reinterpret_cast<const uint4 *>(buf + 16 * (CHUNKS * r + (c ^ ((r >> SH) & (CHUNKS - 1)))));
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) put(PER * i + lane / CHUNKS, lane % CHUNKS, v[i]);
}

template <int T>
__device__ __forceinline__ uint32_t word_of(const float *v) {
    if constexpr (T == QMM_F32) return __float_as_uint(v[0]);
    else if constexpr (T == QMM_F16) {
        const __half2 h = __floats2half2_rn(v[0], v[1]);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[0], v[1]);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

// OWN columns from n0 of the warp's rows, row 0 at element `base` of y, rows
// below `live` only, columns below N only.
template <int T, int CHUNKS, int OWN>
__device__ __forceinline__ void store_tile(uint8_t *buf, int lane, const float (&acc)[OWN], void *y, int64_t base,
                                           int64_t ldy, int live, int n0, int N, bool vec) {
    constexpr int ES = T == QMM_F32 ? 4 : 2, PER = 16 / ES, PW = 4 / ES;  // values per chunk and per word
#pragma unroll
    for (int g = 0; g < OWN; g += CHUNKS * PER) {
        uint4 w[CHUNKS];
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c) {
            const float *v = acc + g + c * PER;
            w[c] = make_uint4(word_of<T>(v), word_of<T>(v + PW), word_of<T>(v + 2 * PW), word_of<T>(v + 3 * PW));
        }
        rows_out<CHUNKS>(buf, lane, w, [&](int r, int c, const uint4 &d) {
            const int n = n0 + g + c * PER;
            if (r >= live || n >= N) return;
            uint8_t *p = static_cast<uint8_t *>(y) + (base + r * ldy + g + c * PER) * ES;
            if (vec && n + PER <= N) {
                *reinterpret_cast<uint4 *>(p) = d;
                return;
            }
            const uint32_t q[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (n + i < N) {
                    if constexpr (ES == 4) reinterpret_cast<uint32_t *>(p)[i] = q[i];
                    else reinterpret_cast<uint16_t *>(p)[i] = static_cast<uint16_t>(q[i >> 1] >> (16 * (i & 1)));
                }
        });
    }
}

// A piece of work, and when it is part of a cut tile the CTAs (or pairs) that
// share the tile (else c0 < 0).
struct Cut {
    int e, nblk, row0, ntok, k0, k1, c0, c1;
};

template <int CG, bool DUAL>
__global__ void __launch_bounds__(Wide<CG, DUAL>::THREADS, 1)
    f8_wide_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmW2,
                   const __grid_constant__ CUtensorMap tmX, const Params P) {
    using C = Wide<CG, DUAL>;
    constexpr int NA = DUAL ? 2 : 1;
    constexpr int PARTS = C::PARTS, EPI = C::EPI, EPI_THREADS = C::EPI_THREADS, OWN = C::OWN, CHUNKS = C::CHUNKS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = CG == 2 ? static_cast<int>(cluster_rank()) : 0;

    const uint32_t stage0 = smem_u32(smem);
    const uint32_t bar = smem_u32(smem + C::OFF_BAR);
    const uint32_t full = bar, empty = full + 8 * C::STAGES;
    const uint32_t d_full = empty + 8 * C::STAGES, d_empty = d_full + 16, done = d_empty + 16;
    const uint32_t sc_full = done + 8, sc_empty = sc_full + 8 * SC_RING;
    const uint32_t pc_full = sc_empty + 8 * SC_RING, pc_empty = pc_full + 8 * PIECES;
    int4 *pieces = reinterpret_cast<int4 *>(smem + C::OFF_PIECES);  // three words of 16 bytes each
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_BAR + 480);
    volatile unsigned *arrived = reinterpret_cast<volatile unsigned *>(smem + C::OFF_BAR + 488);
    int *cum = reinterpret_cast<int *>(smem + C::OFF_CUM);

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(full + 8 * s, 1);
            mbar_init(empty + 8 * s, 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(d_full + 8 * s, 1);
            mbar_init(d_empty + 8 * s, EPI * CG);
        }
        for (int s = 0; s < SC_RING; ++s) {
            mbar_init(sc_full + 8 * s, 32);
            mbar_init(sc_empty + 8 * s, EPI);
        }
        for (int s = 0; s < PIECES; ++s) {
            mbar_init(pc_full + 8 * s, 1);
            mbar_init(pc_empty + 8 * s, 2 + (rank == 0) + EPI);  // copies, scales, MMA, epilogue warps
        }
        mbar_init(done, 1);
        fence_mbar_init();
    }
    if (warp == 3) {
        if constexpr (CG == 1) {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot))
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot))
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        }
    }
    if (warp == 0) count_tiles(cum, P.offsets, P.E, P.R, TOK * CG, P.tiles_n, lane, P.status);
    tc_fence_before();
    __syncthreads();
    if constexpr (CG == 2) cluster_sync();  // the other CTA's barriers are ready
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    // The next piece, from the scheduling warp: the arithmetic that finds it
    // (divisions, a search over the experts, reads of the offsets) is done ahead
    // of the roles and out of their registers.  False after the last one, or
    // when the wait ran out.  With `whole_warp` the caller's lanes are together
    // and the first arrives for them.
    Cut p;
    int np = 0;
    auto next_piece = [&](bool whole_warp) -> bool {
        const int s = np % PIECES;
        bool ok = mbar_spin(pc_full + 8 * s, (np / PIECES) & 1, P.status);
        if (whole_warp) ok = __all_sync(0xffffffffu, ok);
        if (!ok) return false;
        const int4 a = pieces[3 * s], b = pieces[3 * s + 1], c = pieces[3 * s + 2];
        p.row0 = a.x, p.ntok = a.y, p.nblk = a.z, p.e = a.w;
        p.k0 = b.x, p.k1 = b.y, p.c0 = b.z, p.c1 = b.w;
        if (whole_warp) __syncwarp();
        if (!whole_warp || lane == 0) mbar_arrive(pc_empty + 8 * s);
        ++np;
        return c.x != 0;
    };

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_LOW));
        if (warp == 0 && elect_one()) {
            const int stop = blockIdx.x == 0 ? P.stop : NO_STOP;
            const uint32_t full_lead = CG == 2 ? map_rank(full, 0) : full;
            int it = 0;
            bool ok = true;
            pdl_wait();
            pdl_trigger();
            while (ok && next_piece(false)) {
                const int tok = p.row0 + rank * TOK;
                // weight rows of this CTA: all 256, or its half of them
                const int w0 = p.e * P.N + p.nblk * (DUAL ? 128 : 256);
                for (int k = p.k0; k < p.k1; ++k, ++it) {
                    const int s = it % C::STAGES;
                    if (it >= stop ||
                        (it >= C::STAGES && !mbar_spin(empty + 8 * s, ((it / C::STAGES) - 1) & 1, P.status))) {
                        ok = false;
                        break;
                    }
                    const uint32_t st = stage0 + s * C::STAGE, b = full_lead + 8 * s;
                    if constexpr (CG == 1) {
                        mbar_arrive_expect_tx(full + 8 * s, C::STAGE);
                        tma_2d(st, &tmX, k * BK, tok, b);
                        tma_2d(st + C::A_BYTES, &tmW, k * BK, w0, b);
                        tma_2d(st + C::A_BYTES + 128 * BK, DUAL ? &tmW2 : &tmW, k * BK, DUAL ? w0 : w0 + 128, b);
                    } else {
                        if (rank == 0) mbar_arrive_expect_tx(full + 8 * s, 2 * C::STAGE);
                        tma_2d_pair(st, &tmX, k * BK, tok, b);
                        tma_2d_pair(st + C::A_BYTES, &tmW, k * BK, rank ? w0 + 128 : w0, b);
                    }
                }
            }
            // no CTA ends with copies in flight.  The second CTA's complete on the
            // first one's barriers: when every wait succeeded they have landed once
            // the last MMA is done; otherwise it pauses for far longer than a copy
            // takes.
            if (rank == 0) {
                for (int i = it > C::STAGES ? it - C::STAGES : 0; i < it; ++i)
                    mbar_spin(full + 8 * (i % C::STAGES), (i / C::STAGES) & 1, P.status);
            } else if (!ok) {
                const long long t0 = clock64();
                while (clock64() - t0 < DRAIN_CYCLES) __nanosleep(1000);
            }
        } else if (warp == 1 && rank == 0 && elect_one()) {
            int it = 0;
            bool ok = true;
            const uint32_t idesc = (1u << 4) | ((COLS >> 3) << 17) | ((TOK * CG >> 4) << 24);
            while (ok && next_piece(false)) {
                for (int k = p.k0; k < p.k1; ++k, ++it) {
                    const int s = it % C::STAGES, d = it & 1;
                    if (!mbar_spin(full + 8 * s, (it / C::STAGES) & 1, P.status) ||
                        (it >= 2 && !mbar_spin(d_empty + 8 * d, ((it >> 1) - 1) & 1, P.status))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t a = smem_desc(stage0 + s * C::STAGE), b = smem_desc(stage0 + s * C::STAGE + C::A_BYTES);
#pragma unroll
                    for (int q = 0; q < BK / 32; ++q)
                        mma_wide<CG>(tmem + d * COLS, a + 2 * q, b + 2 * q, idesc, q ? 1u : 0u);
                    commit<CG>(empty + 8 * s);
                    commit<CG>(d_full + 8 * d);
                }
            }
            commit<CG>(done);
        } else if (warp == 2) {
            // Scales: xs of this CTA's tokens and the two of W for BATCH K blocks
            // at a time, by asynchronous copies straight into shared memory.
            pdl_wait();
            int ib = 0;
            bool ok = true;
            while (ok && next_piece(true)) {
                const int tok = rank * TOK;
                const int last = max(p.ntok - 1 - tok, 0);
                const float *w = P.Ws + (static_cast<int64_t>(p.e) * P.nb + (DUAL ? p.nblk : 2 * p.nblk)) * P.kb;
                const float *w2 = DUAL ? P.W2s + (w - P.Ws) : 2 * p.nblk + 1 < P.nb ? w + P.kb : w;
                if (lane == 1) w = w2;
                const float *x = P.xs + p.row0 + (tok < p.ntok ? tok : 0);
                for (int kq = p.k0; kq < p.k1; kq += BATCH, ++ib) {
                    const int s = ib % SC_RING;
                    if (ib >= SC_RING)
                        ok = __all_sync(0xffffffffu, mbar_spin(sc_empty + 8 * s, ((ib / SC_RING) - 1) & 1, P.status));
                    if (!ok) break;
                    uint32_t dst = smem_u32(smem + C::OFF_SC) + s * BATCH * SC_FLOATS * 4;
                    for (int k = kq; k < min(kq + BATCH, p.k1); ++k, dst += SC_FLOATS * 4) {
#pragma unroll
                        for (int i = 0; i < TOK / 32; ++i)
                            copy4(dst + 4 * (lane + 32 * i), x + k * P.ld_s + min(lane + 32 * i, last));
                        if (lane < 2) copy4(dst + 4 * (TOK + lane), w + k);
                    }
                    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(sc_full + 8 * s) : "memory");
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        } else if (warp == 3 && elect_one()) {
            Schedule sch;
            sch.cum = cum;
            sch.offsets = P.offsets;
            sch.E = P.E;
            sch.R = P.R;
            sch.kb = P.kb;
            sch.nb = P.tiles_n;
            sch.G = static_cast<int>(gridDim.x) / CG;
            sch.c = static_cast<int>(blockIdx.x) / CG;
            sch.step = TOK * CG;
            sch.least = LEAST;
            sch.init();
            for (int n = 0;; ++n) {
                Piece q = {};
                const bool more = sch.next(q);
                int c0 = -1, c1 = -1;
                if (more && q.k1 - q.k0 < P.kb) sch.sharers(q.tile, c0, c1);
                const int s = n % PIECES;
                if (n >= PIECES && !mbar_spin(pc_empty + 8 * s, ((n / PIECES) - 1) & 1, P.status)) break;
                pieces[3 * s] = make_int4(q.row0, q.ntok, q.nblk, q.e);
                pieces[3 * s + 1] = make_int4(q.k0, q.k1, c0, c1);
                pieces[3 * s + 2] = make_int4(more, 0, 0, 0);
                mbar_arrive(pc_full + 8 * s);
                if (!more) break;
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REGS_HIGH));
        const int quarter = warp & 3, part = (warp - 4) >> 2;  // TMEM lanes and columns
        const int t = 32 * quarter + lane;                     // this thread's token (TMEM lane)
        // columns: OWN of one matrix, or half as many of gate and the same of up, 128 further
        const uint32_t my_tmem = tmem + (static_cast<uint32_t>(32 * quarter) << 16) + (DUAL ? OWN / 2 : OWN) * part;
        uint8_t *rowbuf = smem + C::OFF_ROWS + (warp - 4) * C::ROWS_BYTES;
        const uint32_t d_empty_lead = CG == 2 ? map_rank(d_empty, 0) : d_empty;
        pdl_wait();
        int it = 0, ib = 0;
        bool ok = true;
        while (ok && next_piece(true)) {
            float acc[OWN];
#pragma unroll
            for (int i = 0; i < OWN; ++i) acc[i] = 0.0f;
            const int tok = rank * TOK + t;  // within the tile
            const bool live = tok < p.ntok;
            for (int kq = p.k0; ok && kq < p.k1; kq += BATCH, ++ib) {
                const int sb = ib % SC_RING;
                ok = __all_sync(0xffffffffu, mbar_spin(sc_full + 8 * sb, (ib / SC_RING) & 1, P.status));
                const float *sc = reinterpret_cast<const float *>(smem + C::OFF_SC) + sb * BATCH * SC_FLOATS;
                const int nk = min(BATCH, p.k1 - kq);
                for (int i = 0; ok && i < nk; ++i, ++it, sc += SC_FLOATS) {
                    const int d = it & 1;
                    float f[NA];
                    f[0] = sc[t] * sc[TOK + (DUAL ? 0 : part * OWN / 128)];
                    if constexpr (DUAL) f[1] = sc[t] * sc[TOK + 1];
                    ok = __all_sync(0xffffffffu, mbar_spin(d_full + 8 * d, (it >> 1) & 1, P.status));
                    if (!ok) break;
                    tc_fence_after();
                    // 16 columns at a time, the next ones on their way meanwhile (the
                    // gated pair: first half gate, second half up)
                    constexpr int NC = OWN / 16;
                    const uint32_t base = my_tmem + d * COLS;
                    auto column = [](int c) { return 16 * c + (DUAL && c >= NC / 2 ? 128 - OWN / 2 : 0); };
                    uint32_t r[2][16];
                    tmem_ld(base, r[0]);
                    tmem_wait(r[0]);
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        if (c + 1 < NC) tmem_ld(base + column(c + 1), r[(c + 1) & 1]);
#pragma unroll
                        for (int j = 0; j < 16; j += 2)
                            fma2(acc[16 * c + j], acc[16 * c + j + 1], r[c & 1][j], r[c & 1][j + 1],
                                 f[DUAL && c >= NC / 2 ? NA - 1 : 0]);
                        if (c + 1 < NC) tmem_wait(r[(c + 1) & 1]);
                        if (c == NC - 2) {
                            // everything is out of this buffer
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) {
                                if constexpr (CG == 2) arrive_cluster(d_empty_lead + 8 * d);
                                else mbar_arrive(d_empty + 8 * d);
                            }
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(sc_empty + 8 * sb);
            }
            // every epilogue warp passes here once per piece, also after a wait
            // that gave up, so that none is left at a barrier alone
            if (named_barrier_or(1, EPI_THREADS, !ok)) {
                ok = false;
                break;
            }
            bool store = true;
            if (p.c0 >= 0) {
                // a part of a cut tile, [groups of 4 columns][128 tokens]
                const int c0 = p.c0, c1 = p.c1;
                const int mine = part * (OWN / 4) * TOK + t;
                float4 *q = reinterpret_cast<float4 *>(P.part + (static_cast<int64_t>(blockIdx.x) * 2 + (p.k0 == 0)) * PART) + mine;
#pragma unroll
                for (int j = 0; j < OWN / 4; ++j)
                    q[j * TOK] = make_float4(acc[4 * j], acc[4 * j + 1], acc[4 * j + 2], acc[4 * j + 3]);
                __threadfence();
                named_barrier(1, EPI_THREADS);
                if (threadIdx.x == 128) *arrived = atomicAdd(P.count + c0 * CG + rank, 1u);
                named_barrier(1, EPI_THREADS);
                store = *arrived == static_cast<unsigned>(c1 - c0);
                if (store) {
                    if (threadIdx.x == 128) P.count[c0 * CG + rank] = 0u;  // zero again for the next launch
                    __threadfence();
#pragma unroll
                    for (int i = 0; i < OWN; ++i) acc[i] = 0.0f;
                    for (int c = c0; c <= c1; ++c) {
                        const float4 *o = reinterpret_cast<const float4 *>(
                                              P.part + ((static_cast<int64_t>(c) * CG + rank) * 2 + (c == c0)) * PART) +
                                          mine;
#pragma unroll
                        for (int j = 0; j < OWN / 4; ++j) {
                            const float4 v = __ldcg(o + j * TOK);
                            acc[4 * j] += v.x;
                            acc[4 * j + 1] += v.y;
                            acc[4 * j + 2] += v.z;
                            acc[4 * j + 3] += v.w;
                        }
                    }
                }
            }
            if (!store) continue;
            const int64_t row0 = p.row0 + rank * TOK + 32 * quarter;  // the warp's first row, and how many it has
            const int rows = p.ntok - rank * TOK - 32 * quarter;
            if constexpr (!DUAL) {
                const int n0 = p.nblk * 256 + OWN * part;
                const int64_t base = row0 * P.ldy + n0;
                if (P.y_type == QMM_F32) store_tile<QMM_F32, CHUNKS>(rowbuf, lane, acc, P.y, base, P.ldy, rows, n0, P.N, P.y_vec);
                else if (P.y_type == QMM_F16) store_tile<QMM_F16, CHUNKS>(rowbuf, lane, acc, P.y, base, P.ldy, rows, n0, P.N, P.y_vec);
                else store_tile<QMM_BF16, CHUNKS>(rowbuf, lane, acc, P.y, base, P.ldy, rows, n0, P.N, P.y_vec);
            } else {
                // h = silu(g) * u; the scale block's largest |h| is over the
                // columns of every warp that shares the token
                uint32_t *amax = reinterpret_cast<uint32_t *>(smem + C::OFF_AMAX);
                constexpr int HC = OWN / 2;  // columns of h per thread
                const int n0 = p.nblk * 128 + HC * part;
                uint32_t a = 0;
#pragma unroll
                for (int i = 0; i < HC; ++i) {
                    const float g = acc[i];
                    const float h = n0 + i < P.N ? silu(g) * acc[HC + i] : 0.0f;
                    acc[i] = h;
                    a = max(a, __float_as_uint(h) & 0x7fffffffu);
                }
                amax[part * TOK + t] = a;
                named_barrier(1, EPI_THREADS);
#pragma unroll
                for (int i = 0; i < PARTS; ++i) a = max(a, amax[i * TOK + t]);
                named_barrier(1, EPI_THREADS);
                float s = __fdiv_rn(__uint_as_float(a), 448.0f);
                s = s < 1.17549435e-38f ? 1.17549435e-38f : s;
                const float inv = __fdiv_rn(1.0f, s);
                if (live && part == 0) P.hs[p.nblk * P.ld_hs + row0 + lane] = s;
                static_assert(HC == 16 * CHUNKS, "one pass of rows_out");
                uint4 w[CHUNKS];
#pragma unroll
                for (int c = 0; c < CHUNKS; ++c) {
                    uint32_t q[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float *v = acc + 16 * c + 4 * i;
                        const uint32_t lo =
                            __nv_cvt_float2_to_fp8x2(make_float2(v[0] * inv, v[1] * inv), __NV_SATFINITE, __NV_E4M3);
                        const uint32_t hi =
                            __nv_cvt_float2_to_fp8x2(make_float2(v[2] * inv, v[3] * inv), __NV_SATFINITE, __NV_E4M3);
                        q[i] = lo | hi << 16;
                    }
                    w[c] = make_uint4(q[0], q[1], q[2], q[3]);
                }
                rows_out<CHUNKS>(rowbuf, lane, w,
                         [&](int r, int c, const uint4 &d) {
                             // (N and the pitch of h are multiples of 16)
                             if (r < rows && n0 + 16 * c < P.N)
                                 *reinterpret_cast<uint4 *>(P.hq + (row0 + r) * P.ld_h + n0 + 16 * c) = d;
                         });
            }
        }
        // Every epilogue warp passes one such barrier per record, the closing
        // record (and one whose wait ran out) too: none is left there alone.
        if (ok) named_barrier_or(1, EPI_THREADS, true);
    }
    tc_fence_before();
    __syncthreads();
    // all MMAs are complete before tensor memory goes (the commits of the
    // pair's MMAs arrive in both CTAs)
    if (warp == 3) {
        mbar_spin(done, 0, P.status);
        tc_fence_after();
    }
    if constexpr (CG == 2) cluster_sync();  // nothing of this CTA is used by the other any more
    if (warp == 3) {
        if constexpr (CG == 1)
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
        else
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

template <int CG, bool DUAL>
cudaError_t launch_wide(const F8Gemm &g, cudaStream_t st, int num_sms) {
    using C = Wide<CG, DUAL>;
    const auto kern = f8_wide_kernel<CG, DUAL>;
    CUtensorMap tw = {}, tw2 = {}, tx = {};
    if (!encode_rows(&tw, g.W, g.E * g.N, g.K, g.K, 128) || (DUAL && !encode_rows(&tw2, g.W2, g.E * g.N, g.K, g.K, 128)) ||
        !encode_rows(&tx, g.xq, g.R, g.K, g.ld_q, TOK))
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
    p.tiles_n = DUAL ? p.nb : (p.nb + 1) / 2;
    p.kb = static_cast<int>(f8_blocks(g.K));
    p.y_type = g.y_type;
    if (!DUAL) {
        const int es = f8_size(g.y_type);
        p.y_vec = reinterpret_cast<uintptr_t>(g.y) % 16 == 0 && g.ldy * es % 16 == 0;
    }
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
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CG;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(num_sms / CG * CG));
    static OncePerDevice ready;
    static std::atomic<int> resident[64];  // CTAs that run at once, per device
    const cudaError_t e = ready(g.dev, [&] {
        cudaError_t r = set_smem_attrs(kern, C::SMEM);
        if (r != cudaSuccess) return r;
        // setmaxnreg draws on what the launch brings: with fewer registers than
        // the split hands out the epilogue would wait for them forever
        cudaFuncAttributes fa;
        if ((r = cudaFuncGetAttributes(&fa, kern)) != cudaSuccess) return r;
        if (fa.numRegs * C::THREADS < 128 * C::REGS_LOW + C::EPI_THREADS * C::REGS_HIGH) return cudaErrorNotSupported;
        int groups = num_sms / CG;
        if (CG == 2) {
            int fit = 0;
            if ((r = cudaOccupancyMaxActiveClusters(&fit, kern, &cfg)) != cudaSuccess) return r;
            if (fit >= 1 && fit < groups) groups = fit;
        }
        resident[g.dev & 63].store(groups * CG);
        return cudaSuccess;
    });
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(static_cast<unsigned>(resident[g.dev & 63].load()));
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, tw, tw2, tx, p);
}

}  // namespace

size_t f8_wide_part_bytes(int num_sms) { return static_cast<size_t>(num_sms) * 2 * PART * sizeof(float); }

cudaError_t launch_f8_wide(const F8Gemm &g, int ctas, cudaStream_t st, int num_sms) {
    if (g.W2) return launch_wide<1, true>(g, st, num_sms);
    return ctas == 2 ? launch_wide<2, false>(g, st, num_sms) : launch_wide<1, false>(g, st, num_sms);
}

}  // namespace qk
