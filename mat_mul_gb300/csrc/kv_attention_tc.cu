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
// 4..7 = conversion of queries, keys and values; 8..11 and 12..15 = rows of
// the first and the second tile (thread = row).
// All waits are bounded: a role whose wait ran out stops, the others' then run
// out too, every copy in flight is waited for and TMEM is freed.
#include "f8_gemm.cuh"
#include "kv_attention.cuh"

namespace qk {
namespace kv {

namespace {

using f8::elect_one;
using f8::mbar_spin;
using f8::tc_fence_after;
using f8::tc_fence_before;

constexpr int TC_THREADS = 512, UNIT = 256;
constexpr int TC_LEAST = 4;  // tiles per CTA below which fewer CTAs take part
constexpr int PIECES = 3, SC_SLOTS = 8, SC_FLOATS = 24;
constexpr float MOVE = 8.0f;      // growth of the maximum that moves the reference
constexpr float TC_SHIFT = 6.0f;  // P as fp16 is at most 2^(MOVE + TC_SHIFT)
constexpr int REGS_A = 56, REGS_B = 56, REGS_C = 200;  // roles 0..3, conversion, rows
static_assert(128 * (REGS_A + REGS_B + 2 * REGS_C) <= 65536, "register split");

template <int DP>
struct Tc {
    static constexpr int ST = 2;               // stages of converted keys and of values
    static constexpr int TILE_BYTES = TILE * DP * 2;  // converted, and one tile of queries
    static constexpr int OFF_K = 2 * TILE_BYTES, OFF_V = OFF_K + ST * TILE_BYTES;
    static constexpr int RAW = TILE * DP;      // codes of a tile
    static constexpr int OFF_RAW = OFF_V + ST * TILE_BYTES;
    static constexpr int OFF_ROW = OFF_RAW + 2 * RAW;             // [2 units] power of two of each row's queries
    static constexpr int OFF_SC = OFF_ROW + 2 * UNIT;              // [SC_SLOTS] key scales, log2 of value scales, their inverses
    static constexpr int OFF_PIECES = OFF_SC + SC_SLOTS * SC_FLOATS * 4;
    static constexpr int OFF_BAR = OFF_PIECES + PIECES * 48;
    static constexpr int SMEM = OFF_BAR + 256 + 1024;
    static_assert(SMEM <= 232448, "shared memory");
    static_assert(2 * RAW >= (TC_THREADS + 1) * 8, "prefix sums lie where the codes will");
    static constexpr int PART = UNIT * (DP + 2);  // floats of a partial result
};

struct TcParams {
    AttnParams a;
    int pairs;  // at most so many (sequence, block of UNIT rows)
    int q_vec, y_vec;
    int stop;
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
__device__ __forceinline__ void tie32(uint32_t *r) {
    asm volatile(""
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
__device__ __forceinline__ void tmem_st16(uint32_t a, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::KV_I4(r, 0),
        KV_I4(r, 4), KV_I4(r, 8), KV_I4(r, 12), "r"(a)
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
    extern __shared__ uint8_t smem_raw[];
    uint8_t *const smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t base = smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    const uint32_t bar = base + C::OFF_BAR;
    const uint32_t raw_full = bar, raw_empty = raw_full + 16;                    // keys, values
    const uint32_t k_full = raw_empty + 16, k_empty = k_full + 8 * C::ST;
    const uint32_t v_full = k_empty + 8 * C::ST, v_empty = v_full + 8 * C::ST;
    const uint32_t q_full = v_empty + 8 * C::ST, q_empty = q_full + 8;
    const uint32_t s_full = q_empty + 8, p_full = s_full + 16, pv_done = p_full + 16, o_empty = pv_done + 16;  // per tile
    const uint32_t pc_full = o_empty + 16, pc_empty = pc_full + 8 * PIECES, done = pc_empty + 8 * PIECES;
    static_assert(32 + 32 * 2 + 16 + 64 + 16 * PIECES + 8 <= 232, "barriers");
    uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_BAR + 232);
    volatile unsigned *const arrived = reinterpret_cast<volatile unsigned *>(smem + C::OFF_BAR + 240);  // per tile
    int4 *const pieces = reinterpret_cast<int4 *>(smem + C::OFF_PIECES);
    int8_t *const row_e = reinterpret_cast<int8_t *>(smem + C::OFF_ROW);
    float *const sc = reinterpret_cast<float *>(smem + C::OFF_SC);
    long long *const pre = reinterpret_cast<long long *>(smem + C::OFF_RAW);

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(raw_full + 8 * i, 1);
            mbar_init(raw_empty + 8 * i, 4);
            mbar_init(s_full + 8 * i, 1);
            mbar_init(p_full + 8 * i, 4);
            mbar_init(pv_done + 8 * i, 1);
            mbar_init(o_empty + 8 * i, 4);
        }
        for (int i = 0; i < C::ST; ++i) {
            mbar_init(k_full + 8 * i, 4);
            mbar_init(k_empty + 8 * i, 1);
            mbar_init(v_full + 8 * i, 4);
            mbar_init(v_empty + 8 * i, 1);
        }
        mbar_init(q_full, 4);
        mbar_init(q_empty, 1);
        for (int i = 0; i < PIECES; ++i) {
            mbar_init(pc_full + 8 * i, 1);
            mbar_init(pc_empty + 8 * i, 1 + 1 + 4 + 8);  // copies, MMA, conversion, rows
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
            int it = 0, issued[2] = {0, 0};
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
                        if (it >= stop) ok = false;
                        if (ok && it > 0) ok = mbar_spin(raw_empty + 8 * side, (it - 1) & 1, P.status);
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
                                d[16] = __fdiv_rn(1.0f, w) * L_FACTOR;
                            }
                            __syncwarp();
                        }
                        if (lane == 0) mbar_arrive_expect_tx(raw_full + 8 * side, bytes);
                        __syncwarp();
                        if (id >= 0)
                            bulk_copy(base + C::OFF_RAW + side * C::RAW + lane * page_bytes, P.codes[side] + tile * page_bytes,
                                      page_bytes, raw_full + 8 * side);
                        issued[side] = it + 1;
                    }
                    if (!ok) break;
                    id = next;
                }
            }
            // no CTA ends with copies in flight
#pragma unroll
            for (int side = 0; side < 2; ++side)
                if (issued[side] > 0) mbar_spin(raw_full + 8 * side, (issued[side] - 1) & 1, P.status);
        } else if (warp == 1 && elect_one()) {
            // ---- MMA issue ----
            constexpr uint32_t ID_S = (1u << 4) | ((TILE >> 3) << 17) | ((128 >> 4) << 24);
            constexpr uint32_t ID_O = (1u << 4) | (1u << 16) | ((DP >> 3) << 17) | ((128 >> 4) << 24);
            int seg = 0, kit = 0, vit = 0, used[2] = {0, 0}, pit[2] = {0, 0};
            bool ok = true;
            auto scores = [&](int t) {
                const uint32_t q = base + t * C::TILE_BYTES, k = base + C::OFF_K + (kit % C::ST) * C::TILE_BYTES;
#pragma unroll
                for (int i = 0; i < KS; ++i) {
                    const uint32_t at = (i >> 2) * (TILE * 128) + 32 * (i & 3);
                    mma_ss(tmem + t * 128, f8::smem_desc(q + at), f8::smem_desc(k + at), ID_S, i ? 1u : 0u);
                }
                commit(s_full + 8 * t);
            };
            auto values = [&](int t, bool first) {
                const uint32_t v = base + C::OFF_V + (vit % C::ST) * C::TILE_BYTES;
#pragma unroll
                for (int i = 0; i < TILE / 16; ++i)
                    mma_ts(tmem + 256 + t * DP, tmem + t * 128 + 8 * i, desc_mn<DP>(v + 2048 * i), ID_O, first && i == 0 ? 0u : 1u);
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
                if (!(ok = mbar_spin(k_full + 8 * (kit % C::ST), (kit / C::ST) & 1, P.status))) break;
                tc_fence_after();
                scores(0);
                if (two) scores(1);
                commit(k_empty + 8 * (kit % C::ST));
                ++kit;
                if (pc.nt == 1) commit(q_empty);
                for (int j = 0; j < pc.nt; ++j) {
                    const bool more = j + 1 < pc.nt;
                    if (!(ok = mbar_spin(v_full + 8 * (vit % C::ST), (vit / C::ST) & 1, P.status))) break;
                    if (!(ok = wait_p(0, j == 0))) break;
                    tc_fence_after();
                    values(0, j == 0);
                    if (more) {
                        if (!(ok = mbar_spin(k_full + 8 * (kit % C::ST), (kit / C::ST) & 1, P.status))) break;
                        tc_fence_after();
                        scores(0);
                    }
                    if (two) {
                        if (!(ok = wait_p(1, j == 0))) break;
                        tc_fence_after();
                        values(1, j == 0);
                    }
                    commit(v_empty + 8 * (vit % C::ST));
                    ++vit;
                    if (more) {
                        if (two) scores(1);
                        commit(k_empty + 8 * (kit % C::ST));
                        ++kit;
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
    } else if (warp < 8) {
        // ---- conversion ----
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_B));
        const int me = tid - 128, w = warp - 4;
        const int cpr = P.dim / 16;  // 16-code chunks of a token
        int it = 0, seg = 0;
        bool ok = true;
        while (ok && next_piece(true)) {
            const int rows = rows_of(), end = end_of(rows);
            // queries: lanes of 8 values, times a power of two that brings a
            // row's largest to [2^13, 2^14)
            if (seg > 0) ok = __all_sync(0xffffffffu, mbar_spin(q_empty, (seg - 1) & 1, P.status));
            if (!ok) break;
            {
                constexpr int LPR = DP / 8, RPW = 32 / LPR, BATCH = 4;
                const int d = 8 * (lane % LPR);
                for (int r = w * RPW + lane / LPR; r < UNIT; r += 4 * RPW * BATCH) {
                    uint4 raw[BATCH];
#pragma unroll
                    for (int k = 0; k < BATCH; ++k) {
                        const int rr = r + k * 4 * RPW;
                        raw[k] = make_uint4(0, 0, 0, 0);
                        if (rr < rows && d < P.dim) {
                            const int qr = pc.r0 + rr, i = qr / P.group;
                            const int64_t at = static_cast<int64_t>(pc.row0 + i) * P.ldq_t +
                                               static_cast<int64_t>(pc.head * P.group + (qr - i * P.group)) * P.ldq_h + d;
                            const uint16_t *src = static_cast<const uint16_t *>(P.q) + at;
                            if (PP.q_vec) raw[k] = __ldg(reinterpret_cast<const uint4 *>(src));
                            else {
                                uint32_t v[8];
#pragma unroll
                                for (int e = 0; e < 8; ++e) v[e] = __ldg(src + e);
                                raw[k] = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
                            }
                        }
                    }
#pragma unroll
                    for (int k = 0; k < BATCH; ++k) {
                        const int rr = r + k * 4 * RPW;
                        const uint32_t x[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
                        float v[8], top = 0.0f;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if (P.q_type == QMM_BF16) {
                                v[2 * e] = __uint_as_float(x[e] << 16), v[2 * e + 1] = __uint_as_float(x[e] & 0xffff0000u);
                            } else {
                                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&x[e]));
                                v[2 * e] = f.x, v[2 * e + 1] = f.y;
                            }
                        }
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float a = fabsf(v[e]);
                            top = a <= 3.402823466e38f ? fmaxf(top, a) : top;
                        }
#pragma unroll
                        for (int o = LPR / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                        const int e2 = top > 0.0f ? min(max(13 - exponent_of(__float_as_uint(top)), -114), 100) : 0;
                        const float up = P.factor < 0.0f ? -pow2f(e2) : pow2f(e2);
                        if (d < P.dim) {
                            const uint4 h = make_uint4(pack_half(v[0] * up, v[1] * up), pack_half(v[2] * up, v[3] * up),
                                                       pack_half(v[4] * up, v[5] * up), pack_half(v[6] * up, v[7] * up));
                            const int t = rr >> 7, tr = rr & 127;
                            *reinterpret_cast<uint4 *>(smem + t * C::TILE_BYTES + (d >> 6) * (TILE * 128) + tr * 128 +
                                                       ((((d & 63) >> 3) ^ (tr & 7)) << 4)) = h;
                        }
                        if (d == 0) row_e[(seg & 1) * UNIT + rr] = static_cast<int8_t>(e2);
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(q_full);
                ++seg;
            }
            for (int j = 0; ok && j < pc.nt; ++j, ++it) {
                const int s = it % C::ST, live = end - (pc.tile + j) * TILE;  // tokens below it are in the sequence
#pragma unroll
                for (int side = 0; side < 2; ++side) {
                    const uint32_t full = side ? v_full : k_full, empty = side ? v_empty : k_empty;
                    bool go = mbar_spin(raw_full + 8 * side, it & 1, P.status);
                    if (go && it >= C::ST) go = mbar_spin(empty + 8 * s, ((it / C::ST) - 1) & 1, P.status);
                    ok = __all_sync(0xffffffffu, go);
                    if (!ok) break;
                    const uint4 *src = reinterpret_cast<const uint4 *>(smem + C::OFF_RAW + side * C::RAW);
                    uint8_t *dst = smem + (side ? C::OFF_V : C::OFF_K) + s * C::TILE_BYTES;
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
#pragma unroll 4
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
                        mbar_arrive(full + 8 * s);
                        mbar_arrive(raw_empty + 8 * side);
                    }
                }
            }
        }
    } else {
        // ---- rows ----
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_C));
        const int t = (warp - 8) >> 2, lane_row = 32 * (warp & 3) + lane;  // tile, and this thread's row (TMEM lane) of it
        const uint32_t my_s = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + t * 128;
        const uint32_t my_o = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + 256 + t * DP;
        int it = 0, tiles = 0, seg = 0;  // tiles of this role, tiles and units of the CTA
        bool ok = true;
        while (ok && next_piece(true)) {
            const int rows = rows_of();
            const int mine = 128 * t + lane_row, start = pc.len - pc.n;
            bool store = false;
            float ref = -INFINITY, l = 0.0f;
            if (rows > 128 * t) {
                // tokens that this row sees, and those that all rows see
                const int i = (pc.r0 + min(mine, rows - 1)) / P.group;
                const int hi = P.causal ? min(pc.len, start + i + 1) : pc.len, lo = P.window ? start + i - P.window + 1 : 0;
                const int first_i = (pc.r0 + 128 * t) / P.group, last_i = (pc.r0 + min(rows, 128 * t + 128) - 1) / P.group;
                const int all_hi = P.causal ? min(pc.len, start + first_i + 1) : pc.len;
                const int all_lo = P.window ? start + last_i - P.window + 1 : 0;
                float f = 0.0f;
                for (int j = 0; j < pc.nt; ++j, ++it) {
                    const float4 *scale = reinterpret_cast<const float4 *>(sc + ((tiles + j) % SC_SLOTS) * SC_FLOATS);
                    ok = __all_sync(0xffffffffu, mbar_spin(s_full + 8 * t, it & 1, P.status));
                    if (!ok) break;
                    tc_fence_after();
                    uint32_t s[TILE];
#pragma unroll
                    for (int k = 0; k < 4; ++k) tmem_ld32(my_s + 32 * k, s + 32 * k);
                    tmem_wait32(s);
                    tie32(s + 32), tie32(s + 64), tie32(s + 96);
                    if (j == 0) f = fabsf(P.factor) * pow2f(-row_e[(seg & 1) * UNIT + mine]);
                    float x[TILE];
#pragma unroll
                    for (int k = 0; k < TILE; ++k) x[k] = __uint_as_float(s[k]);
                    float fs[8], lv[8];
                    {
                        const float4 a = scale[0], b = scale[1], c = scale[2], d = scale[3];
                        fs[0] = f * a.x, fs[1] = f * a.y, fs[2] = f * a.z, fs[3] = f * a.w;
                        fs[4] = f * b.x, fs[5] = f * b.y, fs[6] = f * b.z, fs[7] = f * b.w;
                        lv[0] = c.x, lv[1] = c.y, lv[2] = c.z, lv[3] = c.w, lv[4] = d.x, lv[5] = d.y, lv[6] = d.z, lv[7] = d.w;
                    }
                    const int tok = (pc.tile + j) * TILE;
                    if (tok < all_lo || tok + TILE > all_hi) {
                        const int from = lo - tok, to = hi - tok;
#pragma unroll
                        for (int k = 0; k < TILE; ++k) {
                            const float v = fmaf(x[k], fs[k / 16], lv[k / 16]);
                            x[k] = k >= from && k < to ? v : -INFINITY;
                        }
#pragma unroll
                        for (int k = 0; k < 8; ++k) fs[k] = 1.0f, lv[k] = 0.0f;
                    }
                    float top = -INFINITY;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        float a = x[16 * k];
#pragma unroll
                        for (int e = 1; e < 16; ++e) a = fmaxf(a, x[16 * k + e]);
                        top = fmaxf(top, fmaf(a, fs[k], lv[k]));
                    }
                    const bool move = top > ref + MOVE;
                    if (__any_sync(0xffffffffu, move)) {
                        const float now = move ? ceilf(top) : ref;
                        const float down = move ? ex2(ref - now) : 1.0f;
                        ref = now;
                        l *= down;
                        if (j > 0) {
                            ok = __all_sync(0xffffffffu, mbar_spin(pv_done + 8 * t, (it - 1) & 1, P.status));
                            if (!ok) break;
                            tc_fence_after();
#pragma unroll
                            for (int k = 0; k < DP / 32; ++k) {
                                uint32_t o[32];
                                tmem_ld32(my_o + 32 * k, o);
                                tmem_wait32(o);
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * down);
                                tmem_st32(my_o + 32 * k, o);
                            }
                        }
                    }
                    const float sub = ref == -INFINITY ? 0.0f : ref;
                    const float4 ia = scale[4], ib = scale[5];
                    const float iv[8] = {ia.x, ia.y, ia.z, ia.w, ib.x, ib.y, ib.z, ib.w};
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        uint32_t p[16];
#pragma unroll
                        for (int k = 2 * h; k < 2 * h + 2; ++k) {
                            const float d = lv[k] - sub + TC_SHIFT;
                            float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
                            for (int e = 0; e < 16; e += 2) {
                                float a = x[16 * k + e], b = x[16 * k + e + 1];
                                fma2(a, b, fs[k], d);
                                a = ex2(a), b = ex2(b);
                                add2(s0, s1, a, b);
                                p[8 * (k & 1) + e / 2] = pack_half(a, b);
                            }
                            l = fmaf(s0 + s1, iv[k], l);
                        }
                        tmem_st16(my_s + 16 * h, p);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(p_full + 8 * t);
                }
                if (ok) ok = __all_sync(0xffffffffu, mbar_spin(pv_done + 8 * t, (it - 1) & 1, P.status));
                tc_fence_after();
                store = ok;
            }
            tiles += pc.nt;
            ++seg;
            // every warp of the tile passes here once per piece, also after a wait
            // that gave up, so that none is left at a barrier alone
            if (named_barrier_or(1 + t, 128, !ok)) {
                ok = false;
                break;
            }
            if (!store) continue;
            auto result = [&](int64_t &at, int64_t &row) {
                const int qr = pc.r0 + mine, i = qr / P.group, h = pc.head * P.group + (qr - i * P.group);
                at = static_cast<int64_t>(pc.row0 + i) * P.ldy_t + static_cast<int64_t>(h) * P.ldy_h;
                row = (static_cast<int64_t>(pc.row0) + i) * P.heads * P.group + h;
            };
            auto put = [&](int64_t at, int d, const float *v, int n) {  // n values from d on
                const int es = P.y_type == QMM_F32 ? 4 : 2, per = 16 / es;
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
                (void)per;
            };
            constexpr float LN2 = 0.6931471805599453f, BACK = 20.0f - TC_SHIFT;
            if (pc.c0 < 0) {
                const float inv = l != 0.0f ? L_FACTOR / l : 0.0f;
                int64_t at, row;
                result(at, row);
#pragma unroll
                for (int k = 0; k < DP / 32; ++k) {
                    uint32_t o[32];
                    tmem_ld32(my_o + 32 * k, o);
                    tmem_wait32(o);
                    if (k == DP / 32 - 1) {  // everything is out: the next unit's sums may come
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(o_empty + 8 * t);
                    }
                    float v[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(o[e]) * inv;
                    if (mine < rows) put(at, 32 * k, v, 32);
                }
                if (P.lse && mine < rows) P.lse[row] = l != 0.0f ? (ref + log2f(l) + BACK) * LN2 : -INFINITY;
            } else {
                // a part of a unit: [groups of four columns][row] sums relative to ref, then ref and l
                float *const part = P.part + (static_cast<int64_t>(cta) * 2 + pc.begin) * C::PART;
#pragma unroll
                for (int k = 0; k < DP / 32; ++k) {
                    uint32_t o[32];
                    tmem_ld32(my_o + 32 * k, o);
                    tmem_wait32(o);
                    if (k == DP / 32 - 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(o_empty + 8 * t);
                    }
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        reinterpret_cast<uint4 *>(part)[(8 * k + e / 4) * UNIT + mine] = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                }
                part[DP * UNIT + mine] = ref;
                part[(DP + 1) * UNIT + mine] = l;
                __threadfence();
                named_barrier(1 + t, 128);
                if (tid % 128 == 0) arrived[t] = atomicAdd(P.count + 2 * pc.c0 + t, 1u);
                named_barrier(1 + t, 128);
                if (arrived[t] == static_cast<unsigned>(pc.c1 - pc.c0)) {
                    if (tid % 128 == 0) P.count[2 * pc.c0 + t] = 0u;  // zero again for the next launch
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
                    for (int k = 0; k < DP / 16; ++k) {
                        float v[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) v[e] = 0.0f;
                        for (int c = pc.c0; c <= pc.c1; ++c) {
                            const float4 *q = reinterpret_cast<const float4 *>(part_of(c)) + 4 * k * UNIT + mine;
                            const float w = ex2(__ldcg(part_of(c) + DP * UNIT + mine) - sub) * inv;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float4 o = __ldcg(q + e * UNIT);
                                v[4 * e] = fmaf(o.x, w, v[4 * e]), v[4 * e + 1] = fmaf(o.y, w, v[4 * e + 1]);
                                v[4 * e + 2] = fmaf(o.z, w, v[4 * e + 2]), v[4 * e + 3] = fmaf(o.w, w, v[4 * e + 3]);
                            }
                        }
                        if (mine < rows) put(at, 16 * k, v, 16);
                    }
                    if (P.lse && mine < rows) P.lse[row] = sum != 0.0f ? (top + log2f(sum) + BACK) * LN2 : -INFINITY;
                }
            }
        }
        // (a closing record, and one whose wait ran out, counts as a piece at the barrier above)
        if (ok) named_barrier_or(1 + t, 128, true);
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
        return fa.numRegs * TC_THREADS < 128 * (REGS_A + REGS_B + 2 * REGS_C) ? cudaErrorNotSupported : cudaSuccess;
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
    return a.dim <= 64 ? launch_dp<64>(p, st, num_sms, dev) : launch_dp<128>(p, st, num_sms, dev);
}

}  // namespace kv
}  // namespace qk
