// kv_attention_tc.cu -- attention over the paged 8-bit cache for many query
// rows (prompts, chunks of prompts) on tcgen05, fp16 and bf16 queries, heads
// of up to 128 values.
//
// The formulas are those of kv_attention.cuh.  A unit is 256 query rows (rows
// of the batch times query heads of one cache head, two TMEM tiles of 128)
// over the tokens that some of them see, 128 at a time:
//   S_t [128 rows x 128 tokens] = Q_t K^T        operands in shared memory
//   P_t = 2^(x - reference) as fp16              over S_t's columns in TMEM
//   O_t [128 rows x dim]       += P_t V          A in TMEM, V as it lies in
//                                                the cache (tokens x dim)
// While the tensor cores work on one tile, the other's warps take the
// exponentials.  The codes arrive by bulk copies, page by page, and four warps
// turn them into fp16 (exactly) in the 128-byte swizzle that the products read.
//
// The reference of a row is its running maximum, but only moved when the
// maximum has grown by more than 2^8 of it: fp16 holds P up to 2^14 then, and O
// is scaled anew a few times per row instead of once per tile.
//
// All units' tiles form one list that is cut into equal shares, one per CTA;
// what is cut is joined by the last of its CTAs, in the order of the tokens.
//
// Warp roles: 0 = copies, 1 = MMA issue, 2 = schedule, 3 = tensor memory;
// 4..7 and 8..11 = conversion of keys and of values, both of queries; 12..19
// and 20..27 = rows of the first and the second tile, two threads per row
// (each with half of the tokens, and half of the columns of O).
// All waits are bounded: a role whose wait ran out stops, the others' then run
// out too, every copy in flight is waited for and TMEM is freed.
#include <type_traits>

#include "f8_gemm.cuh"
#include "kv_attention.cuh"

namespace qk {
namespace kv {

namespace {

using f8::elect_one;
using f8::mbar_spin;
using f8::tc_fence_after;
using f8::tc_fence_before;

constexpr int TC_THREADS = 896, UNIT = 256;
constexpr int TC_LEAST = 4;  // tiles per CTA below which fewer CTAs take part
constexpr int PIECES = 2, SC_SLOTS = 4, SC_FLOATS = 16;
// registers per thread at launch, and after the split between roles 0..3, conversion and rows
constexpr int REGS = 72, REGS_A = 48, REGS_B = 64, REGS_C = 80;
static_assert(128 * (REGS_A + 2 * REGS_B + 4 * REGS_C) <= TC_THREADS * REGS, "register split");
constexpr float MOVE = 8.0f;      // growth of the maximum that moves the reference
constexpr float TC_SHIFT = 6.0f;  // P as fp16 is at most 2^(MOVE + TC_SHIFT)

template <int DP>
struct Tc {
    // Converted keys and values take turns in a ring.  Three slots do: a slot is
    // asked for again two products after its last one, about 1000 cycles.
    static constexpr int RING = DP == 128 ? 3 : 4;
    static constexpr int RAW_RING = 4;                // codes on their way, keys and values in turn
    static constexpr int TILE_BYTES = TILE * DP * 2;  // a slot, and one tile of queries
    static constexpr int OFF_RING = 2 * TILE_BYTES;
    static constexpr int RAW = TILE * DP;             // codes of a slot
    static constexpr int OFF_RAW = OFF_RING + RING * TILE_BYTES;
    static constexpr int OFF_ROW = OFF_RAW + RAW_RING * RAW;             // power of two of each row's queries
    static constexpr int OFF_SHARE = OFF_ROW + UNIT;           // [2 halves][UNIT] what the threads of a row tell each other
    static constexpr int OFF_SC = OFF_SHARE + 2 * UNIT * 4;              // [SC_SLOTS] key scales and log2 of value scales
    static constexpr int OFF_PIECES = OFF_SC + SC_SLOTS * SC_FLOATS * 4;
    static constexpr int OFF_BAR = OFF_PIECES + PIECES * 48;
    static constexpr int SMEM = OFF_BAR + 288;
    static_assert(SMEM <= 232448, "shared memory");
    static_assert(RAW_RING * RAW >= (TC_THREADS + 1) * 8, "prefix sums lie where the codes will");
    static constexpr int PART = UNIT * (DP + 2);  // floats of a partial result
};

struct TcParams {
    AttnParams a;
    int pairs;  // at most so many (sequence, block of UNIT rows)
    int q_vec, y_vec;
    int stop;
    uint32_t div_mul, div_shift;  // row / group = row * div_mul >> div_shift for rows below 2^31
};

// A block of UNIT rows of a sequence and its tiles of tokens.
struct Pair {
    int b, row0, n, len, r0, tile, tiles;
};

// Pair p: sequence b has the pairs from offsets[b] group / UNIT + b on, as many as
// its rows need (no sum over the sequences before it).  tiles = 0 where there
// is none; false where the sequence is refused.
__device__ __forceinline__ bool load_pair(const AttnParams &P, int p, Pair &q) {
    auto begin = [&](int b) { return static_cast<int64_t>(P.offsets ? __ldg(P.offsets + b) : b) * P.group / UNIT + b; };
    q.tiles = 0;
    int first = 0, last = P.B - 1;
    while (first < last) {
        const int mid = (first + last + 1) >> 1;
        if (begin(mid) <= p) first = mid;
        else last = mid - 1;
    }
    const int b = first;
    int lo = b, hi = b + 1;
    if (P.offsets) lo = __ldg(P.offsets + b), hi = __ldg(P.offsets + b + 1);
    const int len = __ldg(P.lengths + b);
    if (lo < 0 || hi < lo || hi > P.T || len < 0 || len > static_cast<int64_t>(P.width) * P.page) return false;
    const int64_t r0 = (p - begin(b)) * UNIT, rows = static_cast<int64_t>(hi - lo) * P.group;
    if (r0 < 0 || r0 >= rows) return true;
    q.b = b, q.row0 = lo, q.n = hi - lo, q.len = len;
    q.r0 = static_cast<int>(r0);
    const int start = len - q.n;
    const int i0 = static_cast<int>(r0 / P.group), i1 = static_cast<int>((min(r0 + UNIT, rows) - 1) / P.group);
    const int end = P.causal ? min(len, start + i1 + 1) : len;
    const int from = P.window ? max(0, start + i0 - P.window + 1) : 0;
    q.tile = from / TILE;
    q.tiles = max(1, end > from ? (end + TILE - 1) / TILE - q.tile : 0);
    return true;
}

__device__ __forceinline__ void bulk_copy(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// Values as they lie in the cache, tokens x dim: the N index (dim) runs along
// the rows of 128 swizzled bytes, groups of 64 of it a tile half apart, the K
// index (token) over the rows, groups of eight 1024 bytes apart.
template <int DP>
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr) {
    uint64_t d = static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>((TILE * 128) >> 4) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}

#define KV_R4(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3])
#define KV_RW4(r, i) "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3])
#define KV_I4(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3])
__device__ __forceinline__ void tmem_ld32(uint32_t a, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
        "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : KV_R4(r, 0), KV_R4(r, 4), KV_R4(r, 8), KV_R4(r, 12), KV_R4(r, 16), KV_R4(r, 20), KV_R4(r, 24), KV_R4(r, 28)
        : "r"(a));
}
// Wait for the loads issued; the registers are operands so that no use moves before.
__device__ __forceinline__ void tmem_wait32(uint32_t *r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : KV_RW4(r, 0), KV_RW4(r, 4), KV_RW4(r, 8), KV_RW4(r, 12), KV_RW4(r, 16), KV_RW4(r, 20), KV_RW4(r, 24),
                   KV_RW4(r, 28)
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t a, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::KV_I4(r, 0),
        KV_I4(r, 4), KV_I4(r, 8), KV_I4(r, 12), KV_I4(r, 16), KV_I4(r, 20), KV_I4(r, 24), KV_I4(r, 28), "r"(a)
        : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t a, uint32_t *r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : KV_R4(r, 0), KV_R4(r, 4), KV_R4(r, 8), KV_R4(r, 12)
                 : "r"(a));
}
__device__ __forceinline__ void tmem_wait16(uint32_t *r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : KV_RW4(r, 0), KV_RW4(r, 4), KV_RW4(r, 8), KV_RW4(r, 12) : : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t a, const uint32_t *r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::KV_I4(r, 0), KV_I4(r, 4), "r"(a)
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// (a, b) * (f, f) + (d, d)
__device__ __forceinline__ void fma2(float &a, float &b, float f, float d) {
    asm("{\n\t.reg .b64 p, q, r;\n\t"
        "mov.b64 p, {%0, %1};\n\t"
        "mov.b64 q, {%2, %2};\n\t"
        "mov.b64 r, {%3, %3};\n\t"
        "fma.rn.f32x2 r, p, q, r;\n\t"
        "mov.b64 {%0, %1}, r;\n\t}"
        : "+f"(a), "+f"(b)
        : "f"(f), "f"(d));
}
__device__ __forceinline__ void add2(float &a, float &b, float c, float d) {
    asm("{\n\t.reg .b64 p, q;\n\t"
        "mov.b64 p, {%0, %1};\n\t"
        "mov.b64 q, {%2, %3};\n\t"
        "add.rn.f32x2 p, p, q;\n\t"
        "mov.b64 {%0, %1}, p;\n\t}"
        : "+f"(a), "+f"(b)
        : "f"(c), "f"(d));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ uint32_t pack_half(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// 16 codes as 32 bytes of fp16.
__device__ __forceinline__ void convert16(const uint4 &w, uint4 &a, uint4 &b) {
    a = make_uint4(halves(w.x), halves_hi(w.x), halves(w.y), halves_hi(w.y));
    b = make_uint4(halves(w.z), halves_hi(w.z), halves(w.w), halves_hi(w.w));
}

template <int DP>
__global__ void __launch_bounds__(TC_THREADS, 1) kv_attention_tc_kernel(const TcParams PP) {
    using C = Tc<DP>;
    constexpr int KS = DP / 16;
    const AttnParams &P = PP.a;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    const uint32_t bar = base + C::OFF_BAR;
    const uint32_t raw_full = bar, raw_empty = raw_full + 8 * C::RAW_RING;
    const uint32_t kv_full = raw_empty + 8 * C::RAW_RING, kv_empty = kv_full + 8 * C::RING;
    const uint32_t q_full = kv_empty + 8 * C::RING, q_empty = q_full + 8;
    const uint32_t s_full = q_empty + 8, p_full = s_full + 16, pv_done = p_full + 16, o_empty = pv_done + 16;  // per tile
    const uint32_t pc_full = o_empty + 16, pc_empty = pc_full + 8 * PIECES, done = pc_empty + 8 * PIECES;
    static_assert(16 * (C::RAW_RING + C::RING) + 16 + 64 + 16 * PIECES + 8 <= 264, "barriers");
    uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_BAR + 264);
    volatile unsigned *const arrived = reinterpret_cast<volatile unsigned *>(smem + C::OFF_BAR + 272);  // per tile
    int4 *const pieces = reinterpret_cast<int4 *>(smem + C::OFF_PIECES);
    int8_t *const row_e = reinterpret_cast<int8_t *>(smem + C::OFF_ROW);
    float *const sc = reinterpret_cast<float *>(smem + C::OFF_SC);
    long long *const pre = reinterpret_cast<long long *>(smem + C::OFF_RAW);

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full + 8 * i, 1);
            mbar_init(p_full + 8 * i, 8);
            mbar_init(pv_done + 8 * i, 1);
            mbar_init(o_empty + 8 * i, 8);
        }
        for (int i = 0; i < C::RAW_RING; ++i) {
            mbar_init(raw_full + 8 * i, 1);
            mbar_init(raw_empty + 8 * i, 4);
        }
        for (int i = 0; i < C::RING; ++i) {
            mbar_init(kv_full + 8 * i, 4);
            mbar_init(kv_empty + 8 * i, 1);
        }
        mbar_init(q_full, 8);
        mbar_init(q_empty, 1);
        for (int i = 0; i < PIECES; ++i) {
            mbar_init(pc_full + 8 * i, 1);
            mbar_init(pc_empty + 8 * i, 1 + 1 + 8 + 16);  // copies, MMA, conversion, rows
        }
        mbar_init(done, 1);
        fence_mbar_init();
    }
    if (warp == 3) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (DP > P.dim) {  // columns that no conversion writes
        uint4 *z = reinterpret_cast<uint4 *>(smem);
        for (int i = tid; i < C::OFF_RAW / 16; i += TC_THREADS) z[i] = make_uint4(0, 0, 0, 0);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    pdl_wait();
    pdl_trigger();

    // the tiles of the pairs before each thread's share of them
    const int share = (PP.pairs + TC_THREADS - 1) / TC_THREADS;
    {
        long long sum = 0;
        for (int p = tid * share; p < min(PP.pairs, (tid + 1) * share); ++p) {
            Pair q;
            if (!load_pair(P, p, q)) atomicOr(P.status, STATUS_INDEX);
            sum += q.tiles;
        }
        sum *= P.heads;
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
        if (tid == TC_THREADS - 1) pre[TC_THREADS] = before + incl;
    }
    __syncthreads();
    const long long W = pre[TC_THREADS];
    const int ctas = static_cast<int>(min(static_cast<long long>(gridDim.x), max(1ll, W / TC_LEAST)));
    const int cta = blockIdx.x;
    const bool any = W > 0 && cta < ctas;
    const long long t_begin = any ? cta * W / ctas : 0, t_end = any ? (cta + 1) * W / ctas : 0;
    int share0 = 0;
    long long before0 = 0;
    if (any) {
        int first = 0, last = TC_THREADS - 1;
        while (first < last) {
            const int mid = (first + last + 1) >> 1;
            if (pre[mid] <= t_begin) first = mid;
            else last = mid - 1;
        }
        share0 = first;
        before0 = pre[first];
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    // The next piece of work, from the scheduling warp.
    struct {
        int row0, n, len, r0, head, b, tile, nt, c0, c1, begin;
    } pc;
    int np = 0;
    auto next_piece = [&](bool whole_warp) -> bool {
        const int s = np % PIECES;
        bool ok = mbar_spin(pc_full + 8 * s, (np / PIECES) & 1, P.status);
        if (whole_warp) ok = __all_sync(0xffffffffu, ok);
        if (!ok) return false;
        const int4 a = pieces[3 * s], b = pieces[3 * s + 1], c = pieces[3 * s + 2];
        pc.row0 = a.x, pc.n = a.y, pc.len = a.z, pc.r0 = a.w;
        pc.head = b.x, pc.b = b.y, pc.tile = b.z, pc.nt = b.w;
        pc.c0 = c.x, pc.c1 = c.y, pc.begin = c.z;
        if (whole_warp) __syncwarp();
        if (!whole_warp || lane == 0) mbar_arrive(pc_empty + 8 * s);
        ++np;
        return c.w != 0;
    };
    auto token_of = [&](int row) { return static_cast<int>(static_cast<uint64_t>(row) * PP.div_mul >> PP.div_shift); };
    auto rows_of = [&]() { return static_cast<int>(min(static_cast<int64_t>(UNIT), static_cast<int64_t>(pc.n) * P.group - pc.r0)); };
    // first token that some row of the unit sees, and the end of them
    auto end_of = [&](int rows) {
        return P.causal ? min(pc.len, pc.len - pc.n + (pc.r0 + rows - 1) / P.group + 1) : pc.len;
    };
    auto from_of = [&]() { return P.window ? max(0, pc.len - pc.n + pc.r0 / P.group - P.window + 1) : 0; };

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_A));
        if (warp == 0) {
            // ---- copies ----
            const int pages = TILE / P.page;  // of a tile
            const uint32_t page_bytes = static_cast<uint32_t>(P.page * P.dim);
            const int stop = cta == 0 ? PP.stop : NO_STOP;
            int it = 0, item = 0;  // tiles, and slots filled (keys and values in turn)
            bool ok = true;
            while (ok && next_piece(true)) {
                const int rows = rows_of(), end = end_of(rows), from = from_of();
                const int32_t *tab = P.table + static_cast<int64_t>(pc.b) * P.ld_table;
                auto page_of = [&](int j) {
                    const int tok = (pc.tile + j) * TILE + lane * P.page;
                    int id = -1;
                    if (lane < pages && j < pc.nt && tok < end && tok + P.page > from) {
                        id = __ldg(tab + tok / P.page);
                        if (id < 0 || id >= P.pages) {
                            atomicOr(P.status, STATUS_INDEX);
                            id = -1;
                        }
                    }
                    return id;
                };
                int id = page_of(0);
                for (int j = 0; j < pc.nt; ++j, ++it) {
                    const int next = page_of(j + 1);
                    const int64_t tile = static_cast<int64_t>(max(id, 0)) * P.heads + pc.head;
                    const float ks = __ldg(P.scales[0] + tile), vs = __ldg(P.scales[1] + tile);
                    const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, id >= 0)) * page_bytes;
#pragma unroll
                    for (int side = 0; side < 2; ++side) {
                        const int slot = item % C::RAW_RING;
                        if (it >= stop) ok = false;
                        if (ok && item >= C::RAW_RING) ok = mbar_spin(raw_empty + 8 * slot, ((item / C::RAW_RING) - 1) & 1, P.status);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                        if (side == 0) {
                            // scales of the groups of 16 tokens
                            const int src = 16 * lane / P.page;
                            const float k = __shfl_sync(0xffffffffu, ks, src), v = __shfl_sync(0xffffffffu, vs, src);
                            if (lane < 8) {
                                const float w = fminf(fmaxf(v, 0x1p-100f), 0x1p127f);
                                float *d = sc + (it % SC_SLOTS) * SC_FLOATS + lane;
                                d[0] = fminf(fmaxf(k, 0x1p-126f), 0x1p127f);
                                d[8] = log2f(w);
                            }
                            __syncwarp();
                        }
                        if (lane == 0) mbar_arrive_expect_tx(raw_full + 8 * slot, bytes);
                        __syncwarp();
                        if (id >= 0)
                            bulk_copy(base + C::OFF_RAW + slot * C::RAW + lane * page_bytes, P.codes[side] + tile * page_bytes,
                                      page_bytes, raw_full + 8 * slot);
                        ++item;
                    }
                    if (!ok) break;
                    id = next;
                }
            }
            // no CTA ends with copies in flight
            for (int i = max(0, item - C::RAW_RING); i < item; ++i)
                mbar_spin(raw_full + 8 * (i % C::RAW_RING), (i / C::RAW_RING) & 1, P.status);
        } else if (warp == 1 && elect_one()) {
            // ---- MMA issue ----
            constexpr uint32_t ID_S = (1u << 4) | ((TILE >> 3) << 17) | ((128 >> 4) << 24);
            constexpr uint32_t ID_O = (1u << 4) | (1u << 16) | ((DP >> 3) << 17) | ((128 >> 4) << 24);
            int seg = 0, used[2] = {0, 0}, pit[2] = {0, 0};
            int ki = 0, vi = 1;  // items in the ring: keys even, values odd
            bool ok = true;
            auto slot_of = [&](int item) { return base + C::OFF_RING + (item % C::RING) * C::TILE_BYTES; };
            auto wait_item = [&](int item) { return mbar_spin(kv_full + 8 * (item % C::RING), (item / C::RING) & 1, P.status); };
            auto free_item = [&](int item) { commit(kv_empty + 8 * (item % C::RING)); };
            auto scores = [&](int t) {
                const uint32_t q = base + t * C::TILE_BYTES, k = slot_of(ki);
#pragma unroll
                for (int i = 0; i < KS; ++i) {
                    const uint32_t at = (i >> 2) * (TILE * 128) + 32 * (i & 3);
                    mma_ss(tmem + t * 128, f8::smem_desc(q + at), f8::smem_desc(k + at), ID_S, i ? 1u : 0u);
                }
                commit(s_full + 8 * t);
            };
            auto values = [&](int t, bool first) {
                const uint32_t v = slot_of(vi);
#pragma unroll
                for (int i = 0; i < TILE / 16; ++i)
                    mma_ts(tmem + 256 + t * DP, tmem + t * 128 + 8 * i + (i >= TILE / 32 ? 32 : 0), desc_mn<DP>(v + 2048 * i), ID_O, first && i == 0 ? 0u : 1u);
                commit(pv_done + 8 * t);
            };
            auto wait_p = [&](int t, bool first) {
                if (!mbar_spin(p_full + 8 * t, pit[t] & 1, P.status)) return false;
                ++pit[t];
                if (first) {
                    if (used[t] > 0 && !mbar_spin(o_empty + 8 * t, (used[t] - 1) & 1, P.status)) return false;
                    ++used[t];
                }
                return true;
            };
            while (ok && next_piece(false)) {
                const bool two = rows_of() > 128;
                if (!(ok = mbar_spin(q_full, seg & 1, P.status))) break;
                if (!(ok = wait_item(ki))) break;
                tc_fence_after();
                scores(0);
                if (two) scores(1);
                free_item(ki);
                ki += 2;
                for (int j = 0; j < pc.nt; ++j) {
                    const bool more = j + 1 < pc.nt;
                    if (!(ok = wait_item(vi))) break;
                    if (!(ok = wait_p(0, j == 0))) break;
                    tc_fence_after();
                    values(0, j == 0);
                    if (more) {
                        if (!(ok = wait_item(ki))) break;
                        tc_fence_after();
                        scores(0);
                    }
                    if (two) {
                        if (!(ok = wait_p(1, j == 0))) break;
                        tc_fence_after();
                        values(1, j == 0);
                    }
                    free_item(vi);
                    vi += 2;
                    // (the rows have read what goes with the queries: they have come with P)
                    if (pc.nt == 1) commit(q_empty);
                    if (more) {
                        if (two) scores(1);
                        free_item(ki);
                        ki += 2;
                        if (j + 2 == pc.nt) commit(q_empty);
                    }
                }
                ++seg;
            }
            commit(done);
        } else if (warp == 2 && elect_one()) {
            // ---- schedule ----
            long long t = t_begin, before = before0;
            int p = share0 * share, n = 0;
            Pair q;
            q.tiles = 0;
            long long off = 0;  // of t in the pair
            if (any)
                for (;; ++p) {
                    load_pair(P, p, q);
                    const long long all = static_cast<long long>(q.tiles) * P.heads;
                    if (t < before + all) {
                        off = t - before;
                        break;
                    }
                    before += all;
                }
            for (;; ++n) {
                const bool more = t < t_end;
                const int s = n % PIECES;
                if (n >= PIECES && !mbar_spin(pc_empty + 8 * s, ((n / PIECES) - 1) & 1, P.status)) break;
                if (more) {
                    const int head = static_cast<int>(off / q.tiles), at = static_cast<int>(off - static_cast<long long>(head) * q.tiles);
                    const int nt = static_cast<int>(min(static_cast<long long>(q.tiles - at), t_end - t));
                    const long long u0 = before + static_cast<long long>(head) * q.tiles, u1 = u0 + q.tiles - 1;
                    int c0 = -1, c1 = -1;
                    if (nt < q.tiles) {
                        c0 = static_cast<int>(((u0 + 1) * ctas - 1) / W);
                        c1 = static_cast<int>(((u1 + 1) * ctas - 1) / W);
                    }
                    pieces[3 * s] = make_int4(q.row0, q.n, q.len, q.r0);
                    pieces[3 * s + 1] = make_int4(head, q.b, q.tile + at, nt);
                    pieces[3 * s + 2] = make_int4(c0, c1, at == 0, 1);
                    t += nt, off += nt;
                    if (t < t_end && off == static_cast<long long>(q.tiles) * P.heads) {
                        before += off;
                        off = 0;
                        do load_pair(P, ++p, q);
                        while (q.tiles == 0);
                    }
                } else {
                    pieces[3 * s + 2] = make_int4(0, 0, 0, 0);
                }
                mbar_arrive(pc_full + 8 * s);
                if (!more) break;
            }
        }
    } else if (warp < 12) {
        // ---- conversion ----
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_B));
        const int side = (warp - 4) >> 2, me = tid & 127, w = warp - 4;  // keys or values
        const int cpr = P.dim / 16;                                     // 16-code chunks of a token
        int item = side, seg = 0;
        bool ok = true;
        while (ok && next_piece(true)) {
            const int rows = rows_of(), end = end_of(rows);
            // queries: lanes of 8 values, times a power of two that brings a
            // row's largest to [2^13, 2^14)
            {
                constexpr int LPR = DP / 8, RPW = 32 / LPR, BATCH = 8, NEXT = 8 * RPW;  // rows of a thread are NEXT apart
                const int d = 8 * (lane % LPR);
                for (int r = w * RPW + lane / LPR; r < UNIT; r += NEXT * BATCH) {
                    uint4 raw[BATCH];
                    if (PP.q_vec) {
#pragma unroll
                        for (int k = 0; k < BATCH; ++k) {
                            const int qr = pc.r0 + min(r + k * NEXT, rows - 1), i = token_of(qr);
                            const uint16_t *src = static_cast<const uint16_t *>(P.q) + static_cast<int64_t>(pc.row0 + i) * P.ldq_t +
                                                  static_cast<int64_t>(pc.head * P.group + (qr - i * P.group)) * P.ldq_h;
                            raw[k] = __ldg(reinterpret_cast<const uint4 *>(src + min(d, P.dim - 8)));
                        }
                    } else {
#pragma unroll 1
                        for (int k = 0; k < BATCH; ++k) {
                            const int qr = pc.r0 + min(r + k * NEXT, rows - 1), i = token_of(qr);
                            const uint16_t *src = static_cast<const uint16_t *>(P.q) + static_cast<int64_t>(pc.row0 + i) * P.ldq_t +
                                                  static_cast<int64_t>(pc.head * P.group + (qr - i * P.group)) * P.ldq_h + min(d, P.dim - 8);
                            uint32_t v[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) v[e] = __ldg(src + e);
#pragma unroll
                            for (int e = 0; e < BATCH - 1; ++e) raw[e] = raw[e + 1];
                            raw[BATCH - 1] = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
                        }
                    }
                    // (the last unit's scores are done: its queries may go)
                    if (r < NEXT && seg > 0) ok = __all_sync(0xffffffffu, mbar_spin(q_empty, (seg - 1) & 1, P.status));
                    if (!ok) break;
                    // the largest |value| of a row: in either type it is in the order of the bits
                    const uint32_t inf = P.q_type == QMM_BF16 ? 0x7f80u : 0x7c00u;
                    uint32_t top[BATCH];
#pragma unroll
                    for (int k = 0; k < BATCH; ++k) {
                        const uint32_t m = __vmaxu2(__vmaxu2(raw[k].x & 0x7fff7fffu, raw[k].y & 0x7fff7fffu),
                                                    __vmaxu2(raw[k].z & 0x7fff7fffu, raw[k].w & 0x7fff7fffu));
                        top[k] = max(m & 0xffffu, m >> 16);
                        if (top[k] >= inf) {  // of the finite ones
                            const uint32_t x[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
                            top[k] = 0;
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const uint32_t a = x[e / 2] >> (16 * (e & 1)) & 0x7fffu;
                                top[k] = a < inf ? max(top[k], a) : top[k];
                            }
                        }
                        if (d >= P.dim) top[k] = 0;
                    }
#pragma unroll
                    for (int o = LPR / 2; o; o >>= 1)
#pragma unroll
                        for (int k = 0; k < BATCH; ++k) top[k] = max(top[k], __shfl_xor_sync(0xffffffffu, top[k], o));
#pragma unroll
                    for (int k = 0; k < BATCH; ++k) {
                        const int rr = r + k * NEXT;
                        const uint32_t x[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
                        const float most = P.q_type == QMM_BF16 ? __uint_as_float(top[k] << 16) : half_bits_to_float(top[k]);
                        const int e2 = most > 0.0f ? min(max(13 - exponent_of(__float_as_uint(most)), -114), 100) : 0;
                        // (rows behind the last are zeros; a negative factor goes to the queries)
                        const float up = rr >= rows ? 0.0f : P.factor < 0.0f ? -pow2f(e2) : pow2f(e2);
                        uint32_t h[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float2 v;
                            if (P.q_type == QMM_BF16) v = make_float2(__uint_as_float(x[e] << 16), __uint_as_float(x[e] & 0xffff0000u));
                            else v = __half22float2(*reinterpret_cast<const __half2 *>(&x[e]));
                            h[e] = rr >= rows ? 0 : pack_half(v.x * up, v.y * up);
                        }
                        const int tr = rr & 127;
                        if (d < P.dim)
                            *reinterpret_cast<uint4 *>(smem + (rr >> 7) * C::TILE_BYTES + (d >> 6) * (TILE * 128) + tr * 128 +
                                                       ((((d & 63) >> 3) ^ (tr & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
                        if (d == 0) row_e[rr] = static_cast<int8_t>(e2);
                    }
                }
                if (!ok) break;
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(q_full);
                ++seg;
            }
            for (int j = 0; ok && j < pc.nt; ++j, item += 2) {
                const int live = end - (pc.tile + j) * TILE;  // tokens below it are in the sequence
                {
                    const int raw = item % C::RAW_RING, s = item % C::RING;
                    bool go = mbar_spin(raw_full + 8 * raw, (item / C::RAW_RING) & 1, P.status);
                    if (go && item >= C::RING) go = mbar_spin(kv_empty + 8 * s, ((item / C::RING) - 1) & 1, P.status);
                    ok = __all_sync(0xffffffffu, go);
                    if (!ok) break;
                    const uint4 *src = reinterpret_cast<const uint4 *>(smem + C::OFF_RAW + raw * C::RAW);
                    uint8_t *dst = smem + C::OFF_RING + s * C::TILE_BYTES;
                    auto one = [&](int row, int c, const uint4 &v) {
                        uint4 a, b;
                        convert16(v, a, b);
                        // (odd halves store their second part first: no two of eight lanes on one bank)
                        const int h = c >> 2, q = 2 * (c & 3), x = row & 7;
                        uint8_t *p = dst + h * (TILE * 128) + row * 128;
                        *reinterpret_cast<uint4 *>(p + (((q + (h & 1)) ^ x) << 4)) = h & 1 ? b : a;
                        *reinterpret_cast<uint4 *>(p + (((q + 1 - (h & 1)) ^ x) << 4)) = h & 1 ? a : b;
                    };
                    if (cpr == DP / 16) {
#pragma unroll
                        for (int k = 0; k < DP / 16; ++k) {
                            const int idx = me + 128 * k, row = idx / (DP / 16), c = idx % (DP / 16);
                            uint4 v = src[idx];
                            // (what is not in the sequence may be anything: its probabilities are 0)
                            if (side && row >= live) v = make_uint4(0, 0, 0, 0);
                            one(row, c, v);
                        }
                    } else {
                        for (int k = 0; k < cpr; ++k) {
                            const int idx = me + 128 * k, row = idx / cpr, c = idx - row * cpr;
                            uint4 v = src[idx];
                            if (side && row >= live) v = make_uint4(0, 0, 0, 0);
                            one(row, c, v);
                        }
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(kv_full + 8 * s);
                        mbar_arrive(raw_empty + 8 * raw);
                    }
                }
            }
        }
    } else {
        // ---- rows ----
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_C));
        // tile, half of its tokens (and of O's columns), and this thread's row (TMEM lane)
        const int t = (warp - 12) >> 3, half = (warp - 12) >> 2 & 1, lane_row = 32 * (warp & 3) + lane;
        constexpr int HT = TILE / 2, HD = DP / 2;
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        const uint32_t my_s = tmem + lanes + t * 128 + half * HT, my_p = my_s;  // (P over the scores that this thread has read)
        const uint32_t my_o = tmem + lanes + 256 + t * DP + half * HD;
        const int pair_bar = 1 + 4 * t + (warp & 3);  // of the two warps that share 32 rows
        const int mine = 128 * t + lane_row;
        float *const tell = reinterpret_cast<float *>(smem + C::OFF_SHARE) + half * UNIT + mine;
        const float *const told = reinterpret_cast<const float *>(smem + C::OFF_SHARE) + (half ^ 1) * UNIT + mine;
        int it = 0, tiles = 0;  // tiles of this role, tiles of the CTA
        bool ok = true;
        while (ok && next_piece(true)) {
            const int rows = rows_of();
            const int start = pc.len - pc.n;
            bool store = false;
            float ref = -INFINITY, l = 0.0f;
            if (rows > 128 * t) {
                // tokens that this row sees, and those that all rows see
                const int i = token_of(pc.r0 + min(mine, rows - 1));
                const int hi = P.causal ? min(pc.len, start + i + 1) : pc.len, lo = P.window ? start + i - P.window + 1 : 0;
                const int first_i = token_of(pc.r0 + 128 * t), last_i = token_of(pc.r0 + min(rows, 128 * t + 128) - 1);
                const int all_hi = P.causal ? min(pc.len, start + first_i + 1) : pc.len;
                const int all_lo = P.window ? start + last_i - P.window + 1 : 0;
                float f = 0.0f;
                for (int j = 0; j < pc.nt; ++j, ++it) {
                    // of keys, log2 of values' (groups of 16 tokens)
                    const float *scale = sc + ((tiles + j) % SC_SLOTS) * SC_FLOATS + half * (HT / 16);
                    ok = __all_sync(0xffffffffu, mbar_spin(s_full + 8 * t, it & 1, P.status));
                    tc_fence_after();
                    if (j == 0) f = fabsf(P.factor) * pow2f(-row_e[mine]);
                    const int tok = (pc.tile + j) * TILE + half * HT;
                    const bool masked = tok < all_lo || tok + HT > all_hi;
                    const int from = lo - tok, to = hi - tok;
                    // The scores are read twice, for the maximum and for the
                    // exponentials: all of them do not fit a thread's registers
                    // beside the rest.
                    float top = -INFINITY;
                    auto maximum = [&](auto with_mask) {
                        uint32_t s[32];
#pragma unroll 1
                        for (int h = 0; h < HT / 32; ++h) {
                            tmem_ld32(my_s + 32 * h, s);
                            tmem_wait32(s);
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const float fk = f * scale[2 * h + k], lv = scale[8 + 2 * h + k];
                                float a[16];
#pragma unroll
                                for (int e = 0; e < 16; ++e) {
                                    a[e] = __uint_as_float(s[16 * k + e]);
                                    if constexpr (with_mask.value) {
                                        const int c = 32 * h + 16 * k + e;
                                        a[e] = c >= from && c < to ? fmaf(a[e], fk, lv) : -INFINITY;
                                    }
                                }
                                const float m = max3(max3(max3(a[0], a[1], a[2]), max3(a[3], a[4], a[5]), max3(a[6], a[7], a[8])),
                                                     max3(a[9], a[10], a[11]), max3(max3(a[12], a[13], a[14]), a[15], a[0]));
                                top = fmaxf(top, with_mask.value ? m : fmaf(m, fk, lv));
                            }
                        }
                    };
                    if (ok) {
                        if (masked) maximum(std::true_type());
                        else maximum(std::false_type());
                    }
                    *tell = top;
                    // (both warps of the pair take the same way from here)
                    if (named_barrier_or(pair_bar, 64, !ok)) {
                        ok = false;
                        break;
                    }
                    top = fmaxf(top, *told);
                    const bool move = top > ref + MOVE;
                    if (__any_sync(0xffffffffu, move)) {
                        const float now = move ? ceilf(top) : ref;
                        const float down = move ? ex2(ref - now) : 1.0f;
                        ref = now;
                        l *= down;
                        if (j > 0) {
                            ok = __all_sync(0xffffffffu, mbar_spin(pv_done + 8 * t, (it - 1) & 1, P.status));
                            tc_fence_after();
#pragma unroll 1
                            for (int k = 0; ok && k < HD / 32; ++k) {
                                uint32_t o[32];
                                tmem_ld32(my_o + 32 * k, o);
                                tmem_wait32(o);
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * down);
                                tmem_st32(my_o + 32 * k, o);
                            }
                        }
                    }
                    const float sub = ref == -INFINITY ? 0.0f : ref;  // (a row that has seen nothing yet: any finite one)
                    auto exponentials = [&](auto with_mask) {
                        uint32_t s[2][16];
                        tmem_ld16(my_s, s[0]);
                        tmem_wait16(s[0]);
#pragma unroll
                        for (int h = 0; h < HT / 16; ++h) {
                            if (h + 1 < HT / 16) tmem_ld16(my_s + 16 * (h + 1), s[(h + 1) & 1]);
                            uint32_t p[8];
                            const float fk = f * scale[h], d = scale[8 + h] - sub + TC_SHIFT;
                            float v[16];
#pragma unroll
                            for (int e = 0; e < 16; e += 2) {
                                float a = __uint_as_float(s[h & 1][e]), b = __uint_as_float(s[h & 1][e + 1]);
                                fma2(a, b, fk, d);
                                if constexpr (with_mask.value) {
                                    const int c = 16 * h + e;
                                    a = c >= from && c < to ? a : -INFINITY;
                                    b = c + 1 >= from && c + 1 < to ? b : -INFINITY;
                                }
                                v[e] = ex2(a), v[e + 1] = ex2(b);
                                p[e / 2] = pack_half(v[e], v[e + 1]);
                            }
#pragma unroll
                            for (int o = 8; o >= 2; o >>= 1)
#pragma unroll
                                for (int e = 0; e < o; e += 2) add2(v[e], v[e + 1], v[e + o], v[e + o + 1]);
                            l = fmaf(v[0] + v[1], ex2(-20.0f - scale[8 + h]), l);  // (L_FACTOR / the values' scale)
                            if (h + 1 < HT / 16) tmem_wait16(s[(h + 1) & 1]);
                            tmem_st8(my_p + 8 * h, p);
                        }
                    };
                    if (masked) exponentials(std::true_type());
                    else exponentials(std::false_type());
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(p_full + 8 * t);
                }
                if (ok) ok = __all_sync(0xffffffffu, mbar_spin(pv_done + 8 * t, (it - 1) & 1, P.status));
                tc_fence_after();
                store = ok;
                *tell = l;
            }
            tiles += pc.nt;
            // every warp of the tile passes here once per piece, also after a wait
            // that gave up, so that none is left at a barrier alone
            if (named_barrier_or(9 + t, 256, !ok)) {
                ok = false;
                break;
            }
            if (!store) continue;
            l += *told;
            named_barrier(pair_bar, 64);  // (it is told the next unit's maxima there)
            auto result = [&](int64_t &at, int64_t &row) {
                const int qr = pc.r0 + mine, i = token_of(qr), h = pc.head * P.group + (qr - i * P.group);
                at = static_cast<int64_t>(pc.row0 + i) * P.ldy_t + static_cast<int64_t>(h) * P.ldy_h;
                row = (static_cast<int64_t>(pc.row0) + i) * P.heads * P.group + h;
            };
            auto put = [&](int64_t at, int d, const float *v, int n) {  // n values from d on
                const int es = P.y_type == QMM_F32 ? 4 : 2;
#pragma unroll
                for (int k = 0; k < n; k += 4) {
                    if (d + k >= P.dim) break;
                    if (PP.y_vec && es == 4) {
                        *reinterpret_cast<float4 *>(static_cast<float *>(P.y) + at + d + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
                    } else if (PP.y_vec) {
                        if (k % 8) continue;
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if (P.y_type == QMM_F16) w[e] = pack_half(v[k + 2 * e], v[k + 2 * e + 1]);
                            else {
                                const __nv_bfloat162 b = __floats2bfloat162_rn(v[k + 2 * e], v[k + 2 * e + 1]);
                                w[e] = *reinterpret_cast<const uint32_t *>(&b);
                            }
                        }
                        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(P.y) + at + d + k) = make_uint4(w[0], w[1], w[2], w[3]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) store_typed(P.y, at + d + k + e, P.y_type, v[k + e]);
                    }
                }
            };
            constexpr float LN2 = 0.6931471805599453f, BACK = 20.0f - TC_SHIFT;
            if (pc.c0 < 0) {
                const float inv = l != 0.0f ? L_FACTOR / l : 0.0f;
                int64_t at, row;
                result(at, row);
#pragma unroll
                for (int k = 0; k < HD / 32; ++k) {
                    uint32_t o[32];
                    tmem_ld32(my_o + 32 * k, o);
                    tmem_wait32(o);
                    if (k == HD / 32 - 1) {  // everything is out: the next unit's sums may come
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(o_empty + 8 * t);
                    }
                    float v[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(o[e]) * inv;
                    if (mine < rows) put(at, half * HD + 32 * k, v, 32);
                }
                if (P.lse && half == 0 && mine < rows) P.lse[row] = l != 0.0f ? (ref + log2f(l) + BACK) * LN2 : -INFINITY;
            } else {
                // a part of a unit: [groups of four columns][row] sums relative to ref, then ref and l
                float *const part = P.part + (static_cast<int64_t>(cta) * 2 + pc.begin) * C::PART;
#pragma unroll
                for (int k = 0; k < HD / 32; ++k) {
                    uint32_t o[32];
                    tmem_ld32(my_o + 32 * k, o);
                    tmem_wait32(o);
                    if (k == HD / 32 - 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(o_empty + 8 * t);
                    }
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        reinterpret_cast<uint4 *>(part)[(half * HD / 4 + 8 * k + e / 4) * UNIT + mine] = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                }
                if (half == 0) part[DP * UNIT + mine] = ref, part[(DP + 1) * UNIT + mine] = l;
                __threadfence();
                named_barrier(9 + t, 256);
                if ((warp - 12) % 8 == 0 && lane == 0) arrived[t] = atomicAdd(P.count + 2 * pc.c0 + t, 1u);
                named_barrier(9 + t, 256);
                if (arrived[t] == static_cast<unsigned>(pc.c1 - pc.c0)) {
                    if ((warp - 12) % 8 == 0 && lane == 0) P.count[2 * pc.c0 + t] = 0u;  // zero again for the next launch
                    __threadfence();
                    auto part_of = [&](int c) { return P.part + (static_cast<int64_t>(c) * 2 + (c == pc.c0)) * C::PART; };
                    float top = -INFINITY, sum = 0.0f;
                    for (int c = pc.c0; c <= pc.c1; ++c) top = fmaxf(top, __ldcg(part_of(c) + DP * UNIT + mine));
                    const float sub = top == -INFINITY ? 0.0f : top;
                    for (int c = pc.c0; c <= pc.c1; ++c)
                        sum = fmaf(__ldcg(part_of(c) + (DP + 1) * UNIT + mine), ex2(__ldcg(part_of(c) + DP * UNIT + mine) - sub), sum);
                    const float inv = sum != 0.0f ? L_FACTOR / sum : 0.0f;
                    int64_t at, row;
                    result(at, row);
#pragma unroll 1
                    for (int k = half * HD / 32; k < (half + 1) * HD / 32; ++k) {
                        float v[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] = 0.0f;
#pragma unroll 1
                        for (int c = pc.c0; c <= pc.c1; ++c) {
                            const float4 *q = reinterpret_cast<const float4 *>(part_of(c)) + 8 * k * UNIT + mine;
                            const float w = ex2(__ldcg(part_of(c) + DP * UNIT + mine) - sub) * inv;
                            float4 o[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) o[e] = __ldcg(q + e * UNIT);
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                v[4 * e] = fmaf(o[e].x, w, v[4 * e]), v[4 * e + 1] = fmaf(o[e].y, w, v[4 * e + 1]);
                                v[4 * e + 2] = fmaf(o[e].z, w, v[4 * e + 2]), v[4 * e + 3] = fmaf(o[e].w, w, v[4 * e + 3]);
                            }
                        }
                        if (mine < rows) put(at, 32 * k, v, 32);
                    }
                    if (P.lse && half == 0 && mine < rows) P.lse[row] = sum != 0.0f ? (top + log2f(sum) + BACK) * LN2 : -INFINITY;
                }
            }
        }
        // (a closing record, and one whose wait ran out, counts as a piece at the barrier above)
        if (ok) named_barrier_or(9 + t, 256, true);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 3) {
        mbar_spin(done, 0, P.status);  // all MMAs are complete before tensor memory goes
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

template <int DP>
cudaError_t launch_dp(const TcParams &p, cudaStream_t st, int num_sms, int dev) {
    using C = Tc<DP>;
    const auto kern = kv_attention_tc_kernel<DP>;
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
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(num_sms));
    cfg.blockDim = dim3(TC_THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

size_t tc_part_bytes(int dim, int num_sms) {
    return static_cast<size_t>(num_sms) * 2 * (dim <= 64 ? Tc<64>::PART : Tc<128>::PART) * sizeof(float);
}

cudaError_t launch_tc(const AttnParams &a, int stop, cudaStream_t st, int num_sms, int dev) {
    TcParams p = {};
    p.a = a;
    // a negative factor goes to the queries; one that vanishes would lose the masks
    const float least = 1e-30f;
    if (a.factor > -least && a.factor < least) p.a.factor = a.factor < 0 ? -least : least;
    p.pairs = static_cast<int>(a.T * a.group / UNIT + a.B);
    auto vec = [&](const void *x, int type, int64_t ld_t, int64_t ld_h) {
        const int es = f8_size(type);
        return reinterpret_cast<uintptr_t>(x) % 16 == 0 && (a.T == 1 || ld_t * es % 16 == 0) &&
               (a.heads * a.group == 1 || ld_h * es % 16 == 0);
    };
    p.q_vec = vec(a.q, a.q_type, a.ldq_t, a.ldq_h);
    p.y_vec = vec(a.y, a.y_type, a.ldy_t, a.ldy_h);
    p.stop = stop;
    for (p.div_shift = 31; (int64_t(1) << (p.div_shift - 31)) < a.group;) ++p.div_shift;
    p.div_mul = static_cast<uint32_t>(((uint64_t(1) << p.div_shift) + a.group - 1) / a.group);
    return a.dim <= 64 ? launch_dp<64>(p, st, num_sms, dev) : launch_dp<128>(p, st, num_sms, dev);
}

}  // namespace kv
}  // namespace qk
