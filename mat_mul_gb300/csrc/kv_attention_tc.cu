// kv_attention_tc.cu -- attention over the paged 8-bit cache for many query
// rows (prompts, chunks of prompts) on tcgen05, fp16 and bf16 queries, heads
// of up to 128 values.
//
// The formulas are those of kv_attention.cuh.  A unit is 256 query rows (rows
// of the batch times query heads of one cache head, two TMEM tiles of 128)
// over the tokens that some of them see, 128 at a time:
//   S_t [128 rows x 128 tokens] = Q_t K^T       kind::f8f6f4, both in shared memory
//   P_t = 2^(x - reference) as fp16             over S_t's columns in TMEM
//   O_t [128 rows x dim]       += P_t V         kind::f16, A in TMEM, V as it lies
//                                               in the cache (tokens x dim)
// Keys go from the cache to the tensor cores as they are: TMA brings their codes
// in the 128-byte swizzle, and a query is the sum of 8-bit parts, two for bf16 and
// three for fp16, in a power of two that brings its row's largest value to 2^7 to 2^8.
// The first part is e4m3.  Its 4 bits leave at most half a step, 8 units of the last
// of bf16's 8 bits: 3 bits hold that, so the second part is e5m2, whose steps reach
// down to 2^-16 (e4m3's end at 2^-9).  fp16's 11 bits leave 64 units, then 4, and the
// third part is e5m2 as well.  So values down to 2^-6 (at least 2^-13 of the largest)
// are exact; smaller ones are off by at most 2^-14 (bf16) or 2^-17 (fp16), that is
// 2^-21 and 2^-24 of the largest.  Two parts at the rate of 8-bit codes cost what one
// fp16 operand costs.  Values have to meet P in fp16: four warps convert them (exactly).
//
// While the tensor cores work on one tile, the other's warps take the
// exponentials.  The reference of a row is its running maximum, but only moved when
// the maximum has grown by more than 2^8 of it: fp16 holds P up to 2^14 then, and O
// is scaled anew a few times per row instead of once per tile.
//
// All units' tiles form one list that is cut into equal shares, one per CTA, a
// unit counting UNIT_COST tiles more than it has; what is cut is joined by the
// last of its CTAs, in the order of the tokens.
//
// Warp roles: 0 = copies, 1 = MMA issue, 2 = schedule, 3 = tensor memory;
// 4..7 = conversion of values; 8..15 and 16..23 = rows of the first and the
// second tile, two threads per row (each with half of the tokens, and half of the
// columns of O).
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

constexpr int TC_THREADS = 768, UNIT = 256;
constexpr int TC_LEAST = 6;   // tiles (and unit costs) per CTA below which fewer CTAs take part
constexpr int UNIT_COST = 5;  // what a unit costs beside its tiles, in tiles
constexpr int PIECES = 3, SC_SLOTS = 4;
constexpr int SC_FLOATS = 16;  // of 8 groups of tokens: scales of keys (negative: see far_scale), log2 of those of values
// registers per thread at launch, and after the split between roles 0..3, conversion and rows
constexpr int REGS = 80, REGS_A = 48, REGS_B = 48, REGS_C = 96;
static_assert(128 * (REGS_A + REGS_B + 4 * REGS_C) <= TC_THREADS * REGS, "register split");
constexpr float MOVE = 8.0f;      // growth of the maximum that moves the reference
constexpr float TC_SHIFT = 6.0f;  // P as fp16 is at most 2^(MOVE + TC_SHIFT)

// Where P of token group g (16 tokens) of a tile lies, from its first column on:
// over the scores of its thread's half, columns that were read before it is written.
__device__ __forceinline__ constexpr int p_column(int g) { return 64 * (g >> 2) + 32 * (g >> 1 & 1) + 8 * (g & 1); }

// NQ: 8-bit parts of a query.
template <int DP, int NQ>
struct Tc {
    static constexpr int KEYS = TILE * 128;                  // a tile of keys, and a part of a tile of queries: rows of 128 bytes
    static constexpr int KR = DP == 128 && NQ == 3 ? 2 : 4;  // tiles of keys on their way
    static constexpr int VR = 2;                             // tiles of values on their way, and converted
    static constexpr int RAW = TILE * DP, TILE_BYTES = TILE * DP * 2;
    static constexpr int OFF_K = 2 * NQ * KEYS, OFF_V = OFF_K + KR * KEYS, OFF_RAW = OFF_V + VR * TILE_BYTES;
    static constexpr int OFF_SHARE = OFF_RAW + VR * RAW;          // [2 halves][UNIT] what the threads of a row tell each other
    static constexpr int OFF_SC = OFF_SHARE + 2 * UNIT * 4;       // [SC_SLOTS][SC_FLOATS]
    static constexpr int OFF_PIECES = OFF_SC + SC_SLOTS * SC_FLOATS * 4;
    static constexpr int OFF_BAR = OFF_PIECES + PIECES * 48;
    static constexpr int SMEM = OFF_BAR + 320;
    static_assert(SMEM <= 232448, "shared memory");
    static_assert(VR * RAW >= (TC_THREADS + 1) * 8, "prefix sums lie where the codes will");
    static constexpr int PART = UNIT * (DP + 2);  // floats of a partial result
};

struct TcParams {
    AttnParams a;
    int pairs;  // at most so many (sequence, block of UNIT rows)
    int q_vec, y_vec;
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
    const int from = seen_from(P, start + i0);
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
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
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
#define KV_RWF4(m) "+f"(m[0]), "+f"(m[1]), "+f"(m[2]), "+f"(m[3])
#define KV_I4(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3])
__device__ __forceinline__ void tmem_ld16(uint32_t a, uint32_t *r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : KV_R4(r, 0), KV_R4(r, 4), KV_R4(r, 8), KV_R4(r, 12)
                 : "r"(a));
}
// 16 columns and the largest of them.
__device__ __forceinline__ float tmem_max16(uint32_t a, uint32_t *r) {
    float m;
    asm volatile(
        "tcgen05.ld.red.sync.aligned.32x32b.x16.max.f32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, %16, [%17];"
        : KV_R4(r, 0), KV_R4(r, 4), KV_R4(r, 8), KV_R4(r, 12), "=f"(m)
        : "r"(a));
    return m;
}
__device__ __forceinline__ void tmem_wait16(uint32_t *r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : KV_RW4(r, 0), KV_RW4(r, 4), KV_RW4(r, 8), KV_RW4(r, 12) : : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t a, const uint32_t *r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::KV_I4(r, 0), KV_I4(r, 4), "r"(a)
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

// Four values (fp16) as codes, and what the codes leave of them (exact).
template <__nv_fp8_interpretation_t TYPE>
__device__ __forceinline__ uint32_t part4(__half2 (&v)[2]) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const __nv_fp8x2_storage_t c = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(v[i]), __NV_SATFINITE, TYPE);
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(c, TYPE);
        v[i] = __hsub2(v[i], *reinterpret_cast<const __half2 *>(&h));
        w |= static_cast<uint32_t>(c) << (16 * i);
    }
    return w;
}

template <int DP, int NQ>
__global__ void __launch_bounds__(TC_THREADS, 1) kv_attention_tc_kernel(const __grid_constant__ CUtensorMap tmK, const TcParams PP) {
    using C = Tc<DP, NQ>;
    const AttnParams &P = PP.a;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = smem_u32(smem);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

    const uint32_t k_full = base + C::OFF_BAR, k_empty = k_full + 8 * C::KR;
    const uint32_t raw_full = k_empty + 8 * C::KR, raw_empty = raw_full + 8 * C::VR;
    const uint32_t v_full = raw_empty + 8 * C::VR, v_empty = v_full + 8 * C::VR;
    const uint32_t q_full = v_empty + 8 * C::VR, s_full = q_full + 16, pv_done = s_full + 16, o_empty = pv_done + 16;  // per tile
    const uint32_t p_full = o_empty + 16, pc_full = p_full + 16, pc_empty = pc_full + 8 * PIECES, done = pc_empty + 8 * PIECES;
    static_assert(16 * C::KR + 32 * C::VR + 64 + 16 + 16 * PIECES + 8 <= 296, "barriers");
    uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_BAR + 296);
    volatile unsigned *const arrived = reinterpret_cast<volatile unsigned *>(smem + C::OFF_BAR + 304);  // per tile
    volatile unsigned *const nans = arrived + 2;  // a NaN among values that not all rows see, in some unit up to here
    int4 *const pieces = reinterpret_cast<int4 *>(smem + C::OFF_PIECES);
    float *const sc = reinterpret_cast<float *>(smem + C::OFF_SC);
    long long *const pre = reinterpret_cast<long long *>(smem + C::OFF_RAW);

    if (tid == 0) {
        for (int i = 0; i < C::KR; ++i) {
            mbar_init(k_full + 8 * i, 1);
            mbar_init(k_empty + 8 * i, 1);
        }
        for (int i = 0; i < C::VR; ++i) {
            mbar_init(raw_full + 8 * i, 1);
            mbar_init(raw_empty + 8 * i, 4);
            mbar_init(v_full + 8 * i, 4);
            mbar_init(v_empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(q_full + 8 * i, 8);
            mbar_init(s_full + 8 * i, 1);
            mbar_init(pv_done + 8 * i, 1);
            mbar_init(o_empty + 8 * i, 8);
            mbar_init(p_full + 8 * i, 8);
        }
        for (int i = 0; i < PIECES; ++i) {
            mbar_init(pc_full + 8 * i, 1);
            mbar_init(pc_empty + 8 * i, 1 + 1 + 4 + 16);  // copies, MMA, conversion, rows
        }
        mbar_init(done, 1);
        fence_mbar_init();
        *nans = 0;
    }
    if (warp == 3) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    pdl_wait();
    pdl_trigger();

    // what the pairs before each thread's share of them cost
    const int share = (PP.pairs + TC_THREADS - 1) / TC_THREADS;
    {
        long long sum = 0;
        for (int p = tid * share; p < min(PP.pairs, (tid + 1) * share); ++p) {
            Pair q;
            // (offsets that fall can hide a sequence from every search: those of sequence p
            // are looked at by themselves; there are as many pairs as sequences, or more)
            int lo = 0, hi = 0;
            if (P.offsets && p < P.B) lo = __ldg(P.offsets + p), hi = __ldg(P.offsets + p + 1);
            const bool known = load_pair(P, p, q);
            if (!known || lo < 0 || hi < lo || hi > P.T) atomicOr(P.status, STATUS_INDEX);
            if (q.tiles > 0) sum += q.tiles + UNIT_COST;
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
    // (the copies of codes come to where the prefix sums were: by another proxy than these accesses)
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);

    // A piece of work, from the scheduling warp.
    struct Piece {
        int row0, n, len, r0, head, b, tile, nt, c0, c1, begin, more;
    };
    // (volatile: read again where it is needed again, instead of kept in registers)
    auto read_piece = [&](int n) {
        const uint32_t at = base + C::OFF_PIECES + 48 * (n % PIECES);
        Piece p;
        asm volatile("ld.volatile.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(p.row0), "=r"(p.n), "=r"(p.len), "=r"(p.r0) : "r"(at));
        asm volatile("ld.volatile.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(p.head), "=r"(p.b), "=r"(p.tile), "=r"(p.nt) : "r"(at + 16));
        asm volatile("ld.volatile.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(p.c0), "=r"(p.c1), "=r"(p.begin), "=r"(p.more) : "r"(at + 32));
        return p;
    };
    auto piece_bar = [&](int n) { return pc_full + 8 * (n % PIECES); };
    auto piece_parity = [&](int n) { return static_cast<uint32_t>(n / PIECES) & 1; };
    auto free_piece = [&](int n) { mbar_arrive(pc_empty + 8 * (n % PIECES)); };
    // Waits of warps that share a role: the first tests, the others sleep at the
    // named barrier `id` (a testing warp takes eight issue slots per test, which with
    // all of them testing was most of what this kernel executed).  One answer
    // for all of them.
    auto group_wait = [&](bool first, int id, int threads, uint32_t b, uint32_t parity) -> bool {
        bool go = true;
        if (first) go = mbar_spin(b, parity, P.status);
        return !named_barrier_or(id, threads, !go);
    };
    auto token_of = [&](int row) { return kv::token_of(P, row); };
    auto rows_of = [&](const Piece &p) {
        return static_cast<int>(min(static_cast<int64_t>(UNIT), static_cast<int64_t>(p.n) * P.group - p.r0));
    };
    // first token that some row of the unit sees, and the end of them
    auto end_of = [&](const Piece &p) {
        return P.causal ? min(p.len, p.len - p.n + token_of(p.r0 + rows_of(p) - 1) + 1) : p.len;
    };
    // the tokens from one on that all rows of the unit see, and the end of them
    auto all_end_of = [&](const Piece &p) { return P.causal ? min(p.len, p.len - p.n + token_of(p.r0) + 1) : p.len; };
    auto all_from_of = [&](const Piece &p) { return seen_from(P, p.len - p.n + token_of(p.r0 + rows_of(p) - 1)); };
    auto from_of = [&](const Piece &p) { return seen_from(P, p.len - p.n + token_of(p.r0)); };

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_A));
        if (warp == 0) {
            // ---- copies ----
            const int pages = TILE / P.page;  // of a tile
            const uint32_t page_bytes = static_cast<uint32_t>(P.page * P.dim), key_bytes = static_cast<uint32_t>(P.page) * 128;
            const int stop = cta == 0 ? P.stop : NO_STOP;
            int it = 0;
            bool ok = true;
            for (int np = 0; ok; ++np) {
                bool far = false;  // a value scale of the piece, up to here, is far from 1
                ok = __all_sync(0xffffffffu, mbar_spin(piece_bar(np), piece_parity(np), P.status));
                if (!ok) break;
                const Piece pc = read_piece(np);
                __syncwarp();
                if (lane == 0) free_piece(np);
                if (!pc.more) break;
                const int end = end_of(pc), from = from_of(pc);
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
                    const uint32_t live = __popc(__ballot_sync(0xffffffffu, id >= 0));
                    const int k = it % C::KR, v = it % C::VR;
                    if (it >= stop) ok = false;
                    if (ok && it >= C::KR) ok = mbar_spin(k_empty + 8 * k, ((it / C::KR) - 1) & 1, P.status);
                    if (ok && it >= C::VR) ok = mbar_spin(raw_empty + 8 * v, ((it / C::VR) - 1) & 1, P.status);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    // scales of the groups of 16 tokens (the values of tile it - 2 are
                    // converted, so their slot had been freed by tile it - 4, whose
                    // rows are done with the scales that these replace)
                    const int src = 16 * lane / P.page;
                    const float kg = __shfl_sync(0xffffffffu, ks, src), vg = __shfl_sync(0xffffffffu, vs, src);
                    far = far || __any_sync(0xffffffffu, id >= 0 && far_scale(vs));
                    if (lane < 8) {
                        float *d = sc + (it % SC_SLOTS) * SC_FLOATS + lane;
                        const float k = fminf(fmaxf(kg, 0x1p-126f), 0x1p127f);
                        d[0] = far ? -k : k;  // (negative: see far_scale)
                        d[8] = log2f(fminf(fmaxf(vg, 0x1p-100f), 0x1p127f));
                    }
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive_expect_tx(k_full + 8 * k, live * key_bytes);
                        mbar_arrive_expect_tx(raw_full + 8 * v, live * page_bytes);
                    }
                    __syncwarp();
                    if (id >= 0) {
                        tma_page(base + C::OFF_K + k * C::KEYS + lane * key_bytes, &tmK, 0, static_cast<int>(tile), k_full + 8 * k);
                        bulk_copy(base + C::OFF_RAW + v * C::RAW + lane * page_bytes, P.codes[1] + tile * page_bytes, page_bytes,
                                  raw_full + 8 * v);
                    }
                    id = next;
                }
            }
            // no CTA ends with copies in flight
            for (int i = max(0, it - C::KR); i < it; ++i) mbar_spin(k_full + 8 * (i % C::KR), (i / C::KR) & 1, P.status);
            for (int i = max(0, it - C::VR); i < it; ++i) mbar_spin(raw_full + 8 * (i % C::VR), (i / C::VR) & 1, P.status);
        } else if (warp == 1) {
            // ---- MMA issue ----
            // This warp's own instructions were the bottleneck: seven waits, at 300
            // cycles each also where the barrier is complete, and 32 MMAs per tile took
            // 4400 cycles.  Hence one wait for the values and the next keys (the
            // conversion looks after the keys as well), one per tile for P, and a
            // whole warp that stays together, so that the addresses stay in uniform registers.
            constexpr uint32_t ID_S = (1u << 4) | ((TILE >> 3) << 17) | ((128 >> 4) << 24);
            constexpr uint32_t ID_S5 = ID_S | (1u << 7);  // A in e5m2
            constexpr uint32_t ID_O = (1u << 4) | (1u << 16) | ((DP >> 3) << 17) | ((128 >> 4) << 24);
            const uint64_t dq0 = f8::smem_desc(base), dk0 = f8::smem_desc(base + C::OFF_K), dv0 = desc_mn<DP>(base + C::OFF_V);
            const int ks = (P.dim + 31) / 32;
            int units0 = 0, units1 = 0, it0 = 0, it1 = 0;  // of each tile: units with rows in it, P taken
            int ki = 0, vi = 0;
            bool ok = true;
            auto wait = [&](uint32_t b, int phase) { return __all_sync(0xffffffffu, mbar_spin(b, phase & 1, P.status)); };
            auto scores = [&](int t, bool last) {
                const uint64_t dk = dk0 + static_cast<uint64_t>((ki % C::KR) * (C::KEYS >> 4));
                if (elect_one()) {
#pragma unroll
                    for (int n = 0; n < NQ; ++n)
#pragma unroll
                        for (int i = 0; i < DP / 32; ++i)
                            if (i < ks)
                                mma_ss(tmem + t * 128, dq0 + (t * NQ + n) * (C::KEYS >> 4) + 2 * i, dk + 2 * i, n ? ID_S5 : ID_S, n || i ? 1u : 0u);
                    commit(s_full + 8 * t);
                    if (last) commit(k_empty + 8 * (ki % C::KR));
                }
                __syncwarp();
                if (last) ++ki;
            };
            auto values = [&](int t, bool first, bool last) {
                const uint64_t dv = dv0 + static_cast<uint64_t>((vi % C::VR) * (C::TILE_BYTES >> 4));
                if (elect_one()) {
#pragma unroll
                    for (int g = 0; g < TILE / 16; ++g)
                        mma_ts(tmem + 256 + t * DP, tmem + t * 128 + p_column(g), dv + (2048 >> 4) * g, ID_O, first && g == 0 ? 0u : 1u);
                    commit(pv_done + 8 * t);
                    if (last) commit(v_empty + 8 * (vi % C::VR));
                }
                __syncwarp();
                if (last) ++vi;
            };
            for (int np = 0; ok; ++np) {
                if (!(ok = wait(piece_bar(np), np / PIECES))) break;
                const Piece pc = read_piece(np);
                __syncwarp();
                if (lane == 0) free_piece(np);
                const int nt = __shfl_sync(0xffffffffu, pc.more ? pc.nt : 0, 0);
                if (nt == 0) break;
                const bool two = __shfl_sync(0xffffffffu, rows_of(pc) > 128, 0);
                if (!(ok = wait(k_full + 8 * (ki % C::KR), ki / C::KR))) break;
                if (!(ok = wait(q_full, units0++))) break;
                tc_fence_after();
                scores(0, !two);
                if (two) {
                    if (!(ok = wait(q_full + 8, units1++))) break;
                    tc_fence_after();
                    scores(1, true);
                }
                for (int j = 0; j < nt; ++j) {
                    const bool more = j + 1 < nt;
                    if (!(ok = wait(v_full + 8 * (vi % C::VR), vi / C::VR))) break;
                    if (j == 0 && units0 > 1 && !(ok = wait(o_empty, units0))) break;
                    if (!(ok = wait(p_full, it0++))) break;
                    tc_fence_after();
                    values(0, j == 0, !two);
                    if (more) scores(0, !two);
                    if (two) {
                        if (j == 0 && units1 > 1 && !(ok = wait(o_empty + 8, units1))) break;
                        if (!(ok = wait(p_full + 8, it1++))) break;
                        tc_fence_after();
                        values(1, j == 0, true);
                        if (more) scores(1, true);
                    }
                }
            }
            if (elect_one()) commit(done);
            __syncwarp();
        } else if (warp == 2 && elect_one()) {
            // ---- schedule ----
            long long t = t_begin, before = before0;
            int p = share0 * share, n = 0;
            Pair q;
            q.tiles = 0;
            long long off = 0;  // of t in the pair
            auto cost = [&]() { return q.tiles > 0 ? static_cast<long long>(q.tiles + UNIT_COST) * P.heads : 0; };
            if (any)
                for (;; ++p) {
                    load_pair(P, p, q);
                    if (t < before + cost()) {
                        off = t - before;
                        break;
                    }
                    before += cost();
                }
            for (;;) {
                const bool more = t < t_end;
                int at = 0, nt = 0, head = 0, c0 = -1, c1 = -1;
                if (more) {
                    // this CTA's part of the unit: what of its cost is behind UNIT_COST
                    const int all = q.tiles + UNIT_COST;
                    head = static_cast<int>(off / all);
                    const int from = static_cast<int>(off - static_cast<long long>(head) * all);
                    const int to = static_cast<int>(min(static_cast<long long>(all), from + (t_end - t)));
                    at = max(0, from - UNIT_COST);
                    nt = max(0, to - UNIT_COST) - at;
                    if (nt > 0 && nt < q.tiles) {
                        const long long u0 = before + static_cast<long long>(head) * all + UNIT_COST, u1 = u0 + q.tiles - 1;
                        c0 = static_cast<int>(((u0 + 1) * ctas - 1) / W);
                        c1 = static_cast<int>(((u1 + 1) * ctas - 1) / W);
                    }
                    t += to - from, off += to - from;
                }
                if (nt > 0 || !more) {
                    const int s = n % PIECES;
                    if (n >= PIECES && !mbar_spin(pc_empty + 8 * s, ((n / PIECES) - 1) & 1, P.status)) break;
                    pieces[3 * s] = make_int4(q.row0, q.n, q.len, q.r0);
                    pieces[3 * s + 1] = make_int4(head, q.b, q.tile + at, nt);
                    pieces[3 * s + 2] = make_int4(c0, c1, at == 0, more);
                    mbar_arrive(pc_full + 8 * s);
                    ++n;
                }
                if (!more) break;
                if (t < t_end && off == cost()) {
                    before += off;
                    off = 0;
                    do load_pair(P, ++p, q);
                    while (q.tiles == 0);
                }
            }
        }
    } else if (warp < 8) {
        // ---- conversion of values ----
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_B));
        const int me = tid - 128;
        const int cpr = P.dim / 16;  // 16-code chunks of a token
        int it = 0;
        bool ok = true;
        for (int np = 0; ok; ++np) {
            ok = group_wait(warp == 4, 11, 128, piece_bar(np), piece_parity(np));
            if (!ok) break;
            const Piece pc = read_piece(np);
            __syncwarp();
            if (lane == 0) free_piece(np);
            if (!pc.more) break;
            const int end = end_of(pc), from = from_of(pc), all_end = all_end_of(pc), all_from = all_from_of(pc);
            for (int j = 0; j < pc.nt; ++j, ++it) {
                const int tok0 = (pc.tile + j) * TILE;
                const bool whole = tok0 >= all_from && tok0 + TILE <= all_end;
                const int s = it % C::VR, live0 = from - (pc.tile + j) * TILE, live1 = end - (pc.tile + j) * TILE;
                bool go = true;
                if (warp == 4) {
                    go = mbar_spin(raw_full + 8 * s, (it / C::VR) & 1, P.status);
                    if (go && it >= C::VR) go = mbar_spin(v_empty + 8 * s, ((it / C::VR) - 1) & 1, P.status);
                    // (who waits for these values needs the next keys as well)
                    if (go && j + 1 < pc.nt) go = mbar_spin(k_full + 8 * ((it + 1) % C::KR), ((it + 1) / C::KR) & 1, P.status);
                }
                if (named_barrier_or(11, 128, !go)) {
                    ok = false;
                    break;
                }
                uint4 *const src = reinterpret_cast<uint4 *>(smem + C::OFF_RAW + s * C::RAW);
                uint8_t *dst = smem + C::OFF_V + s * C::TILE_BYTES;
                if (!whole) {
                    // (a token that some rows see and some do not: spread_nans)
#pragma unroll 1
                    for (int k = me; k < TILE * cpr; k += 128) {
                        const int row = k / cpr;
                        if (row >= live0 && row < live1 && has_nan(src[k])) src[k] = without_nan(src[k]), *nans = 1;
                    }
                    named_barrier(11, 128);
                }
                auto one = [&](int row, int c, uint4 v) {
                    // (what no row sees may be anything, and is not even there where a
                    // whole page is: its probabilities are 0)
                    if (row < live0 || row >= live1) v = make_uint4(0, 0, 0, 0);
                    uint4 a, b;
                    convert16(v, a, b);
                    // (odd halves store their second part first: no two of eight lanes on one bank)
                    const int h = c >> 2, q = 2 * (c & 3), x = row & 7;
                    uint8_t *p = dst + h * (TILE * 128) + row * 128;
                    *reinterpret_cast<uint4 *>(p + (((q + (h & 1)) ^ x) << 4)) = h & 1 ? b : a;
                    *reinterpret_cast<uint4 *>(p + (((q + 1 - (h & 1)) ^ x) << 4)) = h & 1 ? a : b;
                };
                if (cpr == DP / 16) {
#pragma unroll 1
                    for (int g = 0; g < DP / 16; g += 4) {
                        uint4 v[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) v[k] = src[me + 128 * (g + k)];
#pragma unroll
                        for (int k = 0; k < 4; ++k) one((me + 128 * (g + k)) / (DP / 16), me % (DP / 16), v[k]);
                    }
                } else {
                    for (int k = 0; k < cpr; ++k) {
                        const int idx = me + 128 * k, row = idx / cpr;
                        one(row, idx - row * cpr, src[idx]);
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(v_full + 8 * s);
                    mbar_arrive(raw_empty + 8 * s);
                }
            }
        }
    } else {
        // ---- rows ----
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_C));
        // tile, half of its tokens (and of the row's values), and this thread's row (TMEM lane)
        const int t = (warp - 8) >> 3, half = (warp - 8) >> 2 & 1, lane_row = 32 * (warp & 3) + lane;
        constexpr int HT = TILE / 2, HD = DP / 2;
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        const uint32_t my_s = tmem + lanes + t * 128 + half * HT, my_o = tmem + lanes + 256 + t * DP + half * HD;
        const int pair_bar = 1 + 4 * t + (warp & 3);  // of the two warps that share 32 rows
        const int tile_bar = 9 + t;                   // of the tile's eight
        const bool first = ((warp - 8) & 7) == 0;
        const int mine = 128 * t + lane_row;
        float *const tell = reinterpret_cast<float *>(smem + C::OFF_SHARE) + half * UNIT + mine;
        const volatile float *const told = reinterpret_cast<const float *>(smem + C::OFF_SHARE) + (half ^ 1) * UNIT + mine;
        int it = 0, tiles = 0;  // tiles of this role, tiles of the CTA
        bool ok = true;
        float f = 0.0f;  // scale log2 e over the power of two of the row's queries

        // The queries of piece p as 8-bit parts, in a power of two that brings a row's
        // largest to [2^7, 2^8).  A row goes to DP / 8 lanes, 16 bytes each (with a
        // row per thread every load touched 32 lines: 8000 cycles per unit).
        auto load_queries = [&](const Piece &p) {
            constexpr int LPR = DP / 8, RPW = 32 / LPR, N = 16 / RPW;  // lanes per row, rows per load, loads of a warp's 16 rows
            const int rows = rows_of(p), d = 8 * (lane % LPR);
            const int r0 = 16 * ((warp - 8) & 7) + lane / LPR;  // of the tile's rows, RPW apart
            auto source = [&](int k) {
                const int qr = p.r0 + min(128 * t + r0 + RPW * k, rows - 1), i = token_of(qr);
                return static_cast<const uint16_t *>(P.q) + static_cast<int64_t>(p.row0 + i) * P.ldq_t +
                       static_cast<int64_t>(p.head * P.group + (qr - i * P.group)) * P.ldq_h + min(d, P.dim - 8);
            };
            uint4 raw[N];
            if (PP.q_vec) {  // (all of them on their way at once)
#pragma unroll
                for (int k = 0; k < N; ++k) raw[k] = __ldg(reinterpret_cast<const uint4 *>(source(k)));
            } else {
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    const uint16_t *src = source(k);
                    uint32_t v[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = __ldg(src + e);
                    raw[k] = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
                }
            }
            // the largest |value|: in either type it is in the order of the bits
            constexpr uint32_t INF = NQ == 2 ? 0x7f80u : 0x7c00u;
            uint32_t top[N];
            bool special = false;
#pragma unroll
            for (int k = 0; k < N; ++k) {
                if (r0 + RPW * k + 128 * t >= rows || d >= P.dim) raw[k] = make_uint4(0, 0, 0, 0);
                const uint32_t m = __vmaxu2(__vmaxu2(raw[k].x & 0x7fff7fffu, raw[k].y & 0x7fff7fffu),
                                            __vmaxu2(raw[k].z & 0x7fff7fffu, raw[k].w & 0x7fff7fffu));
                top[k] = max(m & 0xffffu, m >> 16);
                special = special || top[k] >= INF;
            }
            special = __any_sync(0xffffffffu, special);
            if (special) {  // of the finite ones
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    const uint32_t x[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
                    top[k] = 0;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint32_t a = x[e / 2] >> (16 * (e & 1)) & 0x7fffu;
                        top[k] = a < INF ? max(top[k], a) : top[k];
                    }
                }
            }
#pragma unroll
            for (int o = LPR / 2; o; o >>= 1)
#pragma unroll
                for (int k = 0; k < N; ++k) top[k] = max(top[k], __shfl_xor_sync(0xffffffffu, top[k], o));
            float *const factors = reinterpret_cast<float *>(smem + C::OFF_SHARE) + 128 * t;
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const int r = r0 + RPW * k;
                const float most = NQ == 2 ? __uint_as_float(top[k] << 16) : half_bits_to_float(top[k]);
                const int e2 = most > 0.0f ? min(max(7 - exponent_of(__float_as_uint(most)), -120), 100) : 0;
                // (the scores' factor is positive, so that their largest is that of the exponents)
                const float up = P.factor < 0.0f ? -pow2f(e2) : pow2f(e2);
                if (d == 0) factors[r] = fabsf(P.factor) * pow2f(-e2);
                const uint32_t x[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
                uint32_t w[NQ][2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    __half2 v[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t y = x[2 * e + i];
                        float2 z;
                        if constexpr (NQ == 2) z = make_float2(__uint_as_float(y << 16), __uint_as_float(y & 0xffff0000u));
                        else z = __half22float2(*reinterpret_cast<const __half2 *>(&y));
                        z.x *= up, z.y *= up;
                        if (special) {  // (infinities: there is no code)
                            z.x = fabsf(z.x) <= 448.0f ? z.x : __uint_as_float(0x7fffffffu);
                            z.y = fabsf(z.y) <= 448.0f ? z.y : __uint_as_float(0x7fffffffu);
                        }
                        v[i] = __floats2half2_rn(z.x, z.y);
                    }
#pragma unroll
                    for (int n = 0; n < NQ; ++n) w[n][e] = n ? part4<__NV_E5M2>(v) : part4<__NV_E4M3>(v);
                }
#pragma unroll
                for (int n = 0; n < NQ; ++n)
                    *reinterpret_cast<uint2 *>(smem + (t * NQ + n) * C::KEYS + r * 128 + (((d >> 4) ^ (r & 7)) << 4) + (d & 8)) =
                        make_uint2(w[n][0], w[n][1]);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full + 8 * t);
            named_barrier(tile_bar, 256);  // (of all 128 rows)
            f = factors[lane_row];
        };

        int np = 0;
        bool more = false;
        ok = group_wait(first, tile_bar, 256, piece_bar(np), piece_parity(np));
        if (ok) {
            const Piece pc = read_piece(np);
            more = pc.more;
            if (more && rows_of(pc) > 128 * t) load_queries(pc);
        }
        while (ok && more) {
            int tile0, nt, hi, lo, all_hi, all_lo;  // tokens that this row sees, and those that all rows of the unit see
            bool have;                              // rows in this tile
            {
                const Piece pc = read_piece(np);
                const int rows = rows_of(pc);
                have = rows > 128 * t;
                tile0 = pc.tile, nt = pc.nt;
                const int start = pc.len - pc.n, i = token_of(pc.r0 + min(mine, rows - 1));
                hi = P.causal ? min(pc.len, start + i + 1) : pc.len, lo = seen_from(P, start + i);
                all_hi = all_end_of(pc), all_lo = all_from_of(pc);
            }
            float ref = -INFINITY, l = 0.0f;
            FarSum apart;
            bool far = false;
            if (have) {
                int j = 0;
                // (with value scales far from 1 in a loop of its own, as in the other kernels)
#pragma unroll
                for (int mode = 0; mode < 2; ++mode)
                for (; j < nt; ++j, ++it) {
                    if (!ok) break;
                    ok = group_wait(first, tile_bar, 256, s_full + 8 * t, it & 1);
                    if (!ok) break;
                    if (mode == 0 && sc[((tiles + j) % SC_SLOTS) * SC_FLOATS] < 0.0f) break;
                    tc_fence_after();
                    const int tok = (tile0 + j) * TILE;
                    const bool masked = tok < all_lo || tok + TILE > all_hi;  // (as the conversion has it)
                    const int from = lo - tok - half * HT, to = hi - tok - half * HT;
                    // The scores are read twice, for the maximum, which the load itself
                    // finds, and for the exponentials: all of them do not fit a
                    // thread's registers beside the rest.
                    uint32_t s[2][16];
                    float fk[4], lv[4], m[4];  // of the thread's groups of 16 tokens
#pragma unroll
                    for (int h = 0; h < 4; ++h) m[h] = tmem_max16(my_s + 16 * h, s[h & 1]);
                    {
                        const float *scale = sc + ((tiles + j) % SC_SLOTS) * SC_FLOATS + half * 4;
                        const float4 a = *reinterpret_cast<const float4 *>(scale), b = *reinterpret_cast<const float4 *>(scale + 8);
                        fk[0] = f * (mode ? -a.x : a.x), fk[1] = f * (mode ? -a.y : a.y), fk[2] = f * (mode ? -a.z : a.z), fk[3] = f * (mode ? -a.w : a.w);
                        lv[0] = b.x, lv[1] = b.y, lv[2] = b.z, lv[3] = b.w;
                        if (mode == 1) {
                            if (!far) apart.m = ref, apart.l = l;
                            far = true;
#pragma unroll 1
                            for (int k = 0; k < HT; k += 4) {
                                const float factor = f * fabsf(scale[k / 16]);
                                apart.add(4, L_FACTOR * 0x1p6f, [&](int i) {
                                    uint32_t x;
                                    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\ttcgen05.wait::ld.sync.aligned;" : "=r"(x) : "r"(my_s + k + i) : "memory");
                                    return k + i >= from && k + i < to ? __uint_as_float(x) * factor : -INFINITY;
                                });
                            }
                        }
                    }
                    tmem_wait16(s[0]);
                    asm volatile("" : KV_RW4(s[1], 0), KV_RW4(s[1], 4), KV_RW4(s[1], 8), KV_RW4(s[1], 12), KV_RWF4(m) : : "memory");
                    float top = max3(fmaxf(fmaf(m[0], fk[0], lv[0]), fmaf(m[1], fk[1], lv[1])), fmaf(m[2], fk[2], lv[2]),
                                     fmaf(m[3], fk[3], lv[3]));
                    // (the maximum of all tokens will do where it moves nothing)
                    if (masked && __any_sync(0xffffffffu, top > ref + MOVE)) {  // of what the row sees
                        top = -INFINITY;
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            uint32_t r[16];
                            tmem_ld16(my_s + 16 * h, r);
                            tmem_wait16(r);
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const float v = fmaf(__uint_as_float(r[e]), fk[h], lv[h]);
                                top = 16 * h + e >= from && 16 * h + e < to ? fmaxf(top, v) : top;
                            }
                        }
                    }
                    *tell = top;
                    named_barrier(pair_bar, 64);
                    top = fmaxf(top, *told);
                    const bool move = top > ref + MOVE;
                    if (__any_sync(0xffffffffu, move)) {
                        const float now = move ? top : ref;  // (whose P is exact in fp16)
                        const float down = move ? ex2(ref - now) : 1.0f;
                        ref = now;
                        l *= down;
                        if (j > 0) {
                            // (one that runs out has raised the status; the tile's warps go on together)
                            mbar_spin(pv_done + 8 * t, (it - 1) & 1, P.status);
                            __syncwarp();
                            tc_fence_after();
#pragma unroll 1
                            for (int k = 0; k < HD / 16; ++k) {
                                uint32_t o[16];
                                tmem_ld16(my_o + 16 * k, o);
                                tmem_wait16(o);
#pragma unroll
                                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * down);
                                tmem_st16(my_o + 16 * k, o);
                            }
                        }
                    }
                    const float sub = (ref == -INFINITY ? 0.0f : ref) - TC_SHIFT;  // (a row that has seen nothing yet: any finite one)
                    if (masked) {  // (the conversion of the tile's values has looked for NaNs: with_nans reads what it found)
                        const int v = tiles + j;
                        mbar_spin(v_full + 8 * (v % C::VR), (v / C::VR) & 1, P.status);
                        __syncwarp();
                    }
                    // Groups 2 and 3, whose scores are here from the maximum, then 0 and 1.
                    auto exponentials = [&](auto with_mask) {
#pragma unroll
                        for (int i2 = 0; i2 < 4; ++i2) {
                            const int h = (i2 + 2) & 3;
                            uint32_t p[8];
                            float s0 = 0.0f, s1 = 0.0f, s2 = 0.0f, s3 = 0.0f;
#pragma unroll
                            for (int e = 0; e < 16; e += 4) {
                                float a = __uint_as_float(s[i2 & 1][e]), b = __uint_as_float(s[i2 & 1][e + 1]);
                                float c = __uint_as_float(s[i2 & 1][e + 2]), d = __uint_as_float(s[i2 & 1][e + 3]);
                                fma2(a, b, fk[h], lv[h] - sub);
                                fma2(c, d, fk[h], lv[h] - sub);
                                if constexpr (with_mask.value) {
                                    const int k = 16 * h + e;
                                    a = k >= from && k < to ? a : -INFINITY;
                                    b = k + 1 >= from && k + 1 < to ? b : -INFINITY;
                                    c = k + 2 >= from && k + 2 < to ? c : -INFINITY;
                                    d = k + 3 >= from && k + 3 < to ? d : -INFINITY;
                                }
                                a = ex2(a), b = ex2(b), c = ex2(c), d = ex2(d);
                                p[e / 2] = pack_half(a, b), p[e / 2 + 1] = pack_half(c, d);
                                add2(s0, s1, a, b);
                                add2(s2, s3, c, d);
                            }
                            if (i2 < 2) tmem_ld16(my_s + 16 * i2, s[i2 & 1]);
                            l = fmaf(((s0 + s1) + (s2 + s3)) * L_FACTOR, ex2(-lv[h]), l);  // (over the values' scale; 2^-126 at the least)
                            if (i2 == 1 || i2 == 2) tmem_wait16(s[(i2 + 1) & 1]);
                            tmem_st8(my_s + p_column(h), p);
                        }
                    };
                    if (masked) exponentials(std::true_type());
                    else exponentials(std::false_type());
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(p_full + 8 * t);
                }
            }
            tiles += nt;
            // the next piece's queries before this one's results (the tile's warps
            // agree on every wait, also on one that ran out)
            if (ok) ok = group_wait(first, tile_bar, 256, piece_bar(np + 1), piece_parity(np + 1));
            if (!ok) break;
            {
                const Piece next = read_piece(np + 1);
                more = next.more;
                if (more && rows_of(next) > 128 * t) load_queries(next);
            }
            if (have) {
                ok = group_wait(first, tile_bar, 256, pv_done + 8 * t, (it - 1) & 1);
                if (!ok) break;
                tc_fence_after();
                if (far) l = apart.at(ref);
                *tell = l;
                named_barrier(pair_bar, 64);
                l += *told;
                const Piece pc = read_piece(np);
                const int rows = rows_of(pc);
                auto result = [&](int r, int64_t &at, int64_t &row) {
                    const int qr = pc.r0 + r, i = token_of(qr), h = pc.head * P.group + (qr - i * P.group);
                    at = static_cast<int64_t>(pc.row0 + i) * P.ldy_t + static_cast<int64_t>(h) * P.ldy_h;
                    row = (static_cast<int64_t>(pc.row0) + i) * P.heads * P.group + h;
                };
                auto put = [&](int64_t at, int d, const float *v) {  // 16 values from d on
                    if (d >= P.dim) return;
                    if (PP.y_vec && P.y_type == QMM_F32) {
                        float *p = static_cast<float *>(P.y) + at + d;
#pragma unroll
                        for (int k = 0; k < 16; k += 4) *reinterpret_cast<float4 *>(p + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
                    } else if (PP.y_vec) {
                        uint32_t w[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            if (P.y_type == QMM_F16) w[e] = pack_half(v[2 * e], v[2 * e + 1]);
                            else {
                                const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
                                w[e] = *reinterpret_cast<const uint32_t *>(&b);
                            }
                        }
                        uint16_t *p = static_cast<uint16_t *>(P.y) + at + d;
                        if (PP.y_vec == 2) {  // whole sectors of 32 bytes
                            asm volatile("st.global.v8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::KV_I4(w, 0), KV_I4(w, 4), "l"(p)
                                         : "memory");
                        } else {
                            *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
                            *reinterpret_cast<uint4 *>(p + 8) = make_uint4(w[4], w[5], w[6], w[7]);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; ++e) store_typed(P.y, at + d + e, P.y_type, v[e]);
                    }
                };
                // the NaNs among the results that this warp has written, which are its own
                auto with_nans = [&](const auto &set) {
                    __syncwarp();
                    if (__any_sync(0xffffffffu, *nans != 0))
                        spread_nans(P, pc.b, pc.head, pc.len - pc.n, pc.r0, mine - lane, min(rows, mine - lane + 32), half * HD, half * HD + HD,
                                    max(pc.tile * TILE, from_of(pc)), min((pc.tile + pc.nt) * TILE, end_of(pc)), all_from_of(pc), all_end_of(pc),
                                    lane, 32, set);
                };
                constexpr float LN2 = 0.6931471805599453f, BACK = 20.0f - TC_SHIFT;
                if (pc.c0 < 0) {
                    const float inv = l != 0.0f ? L_FACTOR / l : 0.0f;
                    int64_t at, row;
                    result(mine, at, row);
#pragma unroll
                    for (int k = 0; k < HD / 16; ++k) {
                        uint32_t o[16];
                        tmem_ld16(my_o + 16 * k, o);
                        tmem_wait16(o);
                        if (k == HD / 16 - 1) {  // everything is out: the next unit's sums may come
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(o_empty + 8 * t);
                        }
                        float v[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) v[e] = __uint_as_float(o[e]) * inv;
                        if (mine < rows) put(at, half * HD + 16 * k, v);
                    }
                    if (P.lse && half == 0 && mine < rows) P.lse[row] = l != 0.0f ? (ref + log2f(l) + BACK) * LN2 : -INFINITY;
                    with_nans([&](int r, int d) {
                        int64_t y_at, y_row;
                        result(r, y_at, y_row);
                        store_typed(P.y, y_at + d, P.y_type, __uint_as_float(A_NAN));
                    });
                } else {
                    // a part of a unit: [groups of four columns][row] sums relative to ref, then ref and l
                    float *const part = P.part + (static_cast<int64_t>(cta) * 2 + pc.begin) * C::PART;
#pragma unroll
                    for (int k = 0; k < HD / 16; ++k) {
                        uint32_t o[16];
                        tmem_ld16(my_o + 16 * k, o);
                        tmem_wait16(o);
                        if (k == HD / 16 - 1) {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(o_empty + 8 * t);
                        }
#pragma unroll
                        for (int e = 0; e < 16; e += 4)
                            reinterpret_cast<uint4 *>(part)[(half * HD / 4 + 4 * k + e / 4) * UNIT + mine] =
                                make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                    }
                    if (half == 0) part[DP * UNIT + mine] = ref, part[(DP + 1) * UNIT + mine] = l;
                    with_nans([&](int r, int d) { part[(d / 4 * UNIT + r) * 4 + d % 4] = __uint_as_float(A_NAN); });
                    __threadfence();
                    named_barrier(tile_bar, 256);
                    if (first && lane == 0) arrived[t] = atomicAdd(P.count + 2 * pc.c0 + t, 1u + (far ? FAR_PART : 0u));
                    named_barrier(tile_bar, 256);
                    if ((arrived[t] & (FAR_PART - 1)) == static_cast<unsigned>(pc.c1 - pc.c0)) {
                        far = far || arrived[t] >= FAR_PART;  // (of some part: see join_parts)
                        if (first && lane == 0) P.count[2 * pc.c0 + t] = 0u;  // zero again for the next launch
                        __threadfence();
                        auto part_of = [&](int c) { return P.part + (static_cast<int64_t>(c) * 2 + (c == pc.c0)) * C::PART; };
                        float top = -INFINITY, sum = 0.0f;
                        for (int c = pc.c0; c <= pc.c1; ++c) top = fmaxf(top, __ldcg(part_of(c) + DP * UNIT + mine));
                        const float sub = top == -INFINITY ? 0.0f : top;
                        for (int c = pc.c0; c <= pc.c1; ++c)
                            sum = fmaf(__ldcg(part_of(c) + (DP + 1) * UNIT + mine), ex2(__ldcg(part_of(c) + DP * UNIT + mine) - sub), sum);
                        if (far) {
                            sum = 0.0f;
#pragma unroll 1
                            for (int c = pc.c0; c <= pc.c1; ++c)
                                sum += faded(__ldcg(part_of(c) + (DP + 1) * UNIT + mine), __ldcg(part_of(c) + DP * UNIT + mine) - sub);
                        }
                        const float inv = sum != 0.0f ? L_FACTOR / sum : 0.0f;
                        int64_t at, row;
                        result(mine, at, row);
#pragma unroll 1
                        for (int k = half * HD / 16; k < (half + 1) * HD / 16; ++k) {
                            float v[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e) v[e] = 0.0f;
#pragma unroll 2
                            for (int c = pc.c0; c <= pc.c1; ++c) {
                                const float4 *q = reinterpret_cast<const float4 *>(part_of(c)) + 4 * k * UNIT + mine;
                                const float w = ex2(__ldcg(part_of(c) + DP * UNIT + mine) - sub) * inv;
                                float4 o[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e) o[e] = __ldcg(q + e * UNIT);
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    v[4 * e] = fmaf(o[e].x, w, v[4 * e]), v[4 * e + 1] = fmaf(o[e].y, w, v[4 * e + 1]);
                                    v[4 * e + 2] = fmaf(o[e].z, w, v[4 * e + 2]), v[4 * e + 3] = fmaf(o[e].w, w, v[4 * e + 3]);
                                }
                            }
                            if (mine < rows) put(at, 16 * k, v);
                        }
                        if (P.lse && half == 0 && mine < rows) P.lse[row] = sum != 0.0f ? (top + log2f(sum) + BACK) * LN2 : -INFINITY;
                    }
                }
            }
            __syncwarp();
            if (lane == 0) free_piece(np);
            ++np;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 3) {
        mbar_spin(done, 0, P.status);  // all MMAs are complete before tensor memory goes
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

template <int DP, int NQ>
cudaError_t launch_dp(const TcParams &p, cudaStream_t st, int num_sms, int dev) {
    using C = Tc<DP, NQ>;
    const auto kern = kv_attention_tc_kernel<DP, NQ>;
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
    CUtensorMap tm = {};
    if (!encode_pages(&tm, p.a.codes[0], p.a, 128)) return cudaErrorInvalidValue;
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
    return cudaLaunchKernelEx(&cfg, kern, tm, p);
}

}  // namespace

size_t tc_part_bytes(int dim, int num_sms) {
    return static_cast<size_t>(num_sms) * 2 * (dim <= 64 ? Tc<64, 2>::PART : Tc<128, 2>::PART) * sizeof(float);
}

cudaError_t launch_tc(const AttnParams &a, cudaStream_t st, int num_sms, int dev) {
    TcParams p = {};
    p.a = a;
    p.pairs = static_cast<int>(a.T * a.group / UNIT + a.B);
    auto vec = [&](const void *x, int type, int64_t ld_t, int64_t ld_h, int bytes) {
        const int es = f8_size(type);
        return reinterpret_cast<uintptr_t>(x) % bytes == 0 && (a.T == 1 || ld_t * es % bytes == 0) &&
               (a.heads * a.group == 1 || ld_h * es % bytes == 0);
    };
    p.q_vec = vec(a.q, a.q_type, a.ldq_t, a.ldq_h, 16);
    p.y_vec = vec(a.y, a.y_type, a.ldy_t, a.ldy_h, 16) + vec(a.y, a.y_type, a.ldy_t, a.ldy_h, 32);
    if (a.q_type == QMM_BF16) return a.dim <= 64 ? launch_dp<64, 2>(p, st, num_sms, dev) : launch_dp<128, 2>(p, st, num_sms, dev);
    return a.dim <= 64 ? launch_dp<64, 3>(p, st, num_sms, dev) : launch_dp<128, 3>(p, st, num_sms, dev);
}

}  // namespace kv
}  // namespace qk
