// kv_attention_rows.cu -- attention over the paged 8-bit cache for many fp32
// query rows, heads of up to 128 values, on mma.sync.
//
// Formulas, sharing of the work and precision are those of kv_attention.cuh;
// queries and probabilities are the sum of two fp16 values, so every product
// takes two instructions, and these bound it (8 cycles each on a quarter of a
// multiprocessor).  A unit is 128 query rows of one cache head.  Here a warp
// keeps 16 of them to itself, over all tokens:
//   S [16 rows x 128 tokens]  = Q K^T     Q as fragments in shared memory
//   O [16 rows x dim]        += P V       P from the registers that held S
// so nobody exchanges anything, and no warp waits for another but where a row's mask
// cuts a tile.  Every warp converts every code by itself: two conversions per
// four instructions, which the tensor cores' time covers.
//
// Each tile's products with V are summed apart and added with a rounding to
// nearest (the tensor cores cut off what an addition loses).
//
// Measured (1024 rows of 32 heads over 4096 tokens, 8 heads of 128 in the cache):
// 0.32 ms, 371 TFLOP/s of instructions, 62 % of their rate; the kernel that shares a
// tile's tokens between warps took 0.58.  Twelve warps of 152 registers with 32
// or 64 tokens at a time 0.35 to 0.37: a warp's exponentials and conversions are as long
// as its products, and more tokens at a time save more of them than a third warp hides.
#include <type_traits>

#include "kv_attention.cuh"

namespace qk {
namespace kv {

namespace {

// Two warpgroups of rows and one of which a warp brings the tiles; registers per thread
// at launch and after the split.
constexpr int WARPS = 8, ROWS_THREADS = 32 * WARPS + 128;
constexpr int REGS = 168, REGS_COPY = 24, REGS_ROWS = 240;
static_assert(128 * REGS_COPY + 32 * WARPS * REGS_ROWS <= ROWS_THREADS * REGS, "register split");
constexpr int TS = TILE / 16;  // groups of 16 tokens of a tile

template <int DP>
struct Rows {
    static constexpr int R = 16 * WARPS, CONSUMERS = 32 * WARPS, STAGES = 4;
    static constexpr float SHIFT = P_SHIFT;
    static constexpr int ROW = DP == 64 ? 64 : 128, COLS = DP / ROW;
    static constexpr int SIDE = TILE * DP, STAGE = 2 * SIDE;
    static constexpr int OFF_Q = STAGES * STAGE, Q_WARP = DP / 16 * 1024;  // [WARPS][DP / 16][part][lane] fragments
    static constexpr int OFF_SC = OFF_Q + WARPS * Q_WARP;    // [STAGES] scales (as there)
    static constexpr int OFF_BAR = OFF_SC + STAGES * SCALES * 4;
    static constexpr int SMEM = OFF_BAR + 16 * STAGES + 16;
    static_assert(SMEM <= 232448, "shared memory");
    static constexpr int PART = R * (DP + 2);
    static __device__ __forceinline__ int at(int row, int c) {
        if constexpr (DP == 64) return row * 64 + ((c ^ (row >> 1 & 3)) << 4);
        else return row * 128 + ((c ^ (row & 7)) << 4);
    }
};

// Where a CTA's share lies: sequences, blocks of their rows, heads, tiles.  A unit has
// the tiles that its rows see (at least one), so that shares are equal in what there is
// to do; with those of the whole sequence 1024 rows of 4096 tokens took 12 % more.
struct RowWalk {
    int b, block, head, tile;
    int from, tiles;  // of the unit
    long long u0, t;  // tiles before the unit, and before this one
    Seq s;
};

// First token (a multiple of TILE) and tiles of a block of rows.
template <int R>
__device__ __forceinline__ int block_tiles(const AttnParams &P, const Seq &s, int block, int &from) {
    const int start = s.len - s.n;
    const int i0 = token_of(P, block * R), i1 = token_of(P, min(block * R + R, s.n * P.group) - 1);
    const int hi = P.causal ? min(s.len, start + i1 + 1) : s.len;
    from = seen_from(P, start + i0) & ~(TILE - 1);
    return max(1, hi > from ? (hi - from + TILE - 1) / TILE : 0);
}

template <int R>
__device__ __forceinline__ void advance(const AttnParams &P, RowWalk &w, int nt, long long t1) {
    w.t += nt;
    w.tile = 0;
    if (w.t >= t1) return;
    w.u0 += w.tiles;
    if (++w.head < P.heads) return;
    w.head = 0;
    if (++w.block == w.s.blocks) {
        w.block = 0;
        do load_seq<R>(P, ++w.b, w.s);
        while (w.s.units == 0);
    }
    w.tiles = block_tiles<R>(P, w.s, w.block, w.from);
}

template <int R>
__device__ __forceinline__ Span span_of(const AttnParams &P, const RowWalk &w, long long t1) {
    Span u;
    const Seq &s = w.s;
    u.head = w.head;
    u.nt = w.tiles <= SHORT ? w.tiles : static_cast<int>(min(static_cast<long long>(w.tiles - w.tile), t1 - w.t));
    u.r0 = w.block * R;
    u.rows = min(R, s.n * P.group - u.r0);
    const int start = s.len - s.n, i0 = token_of(P, u.r0), i1 = token_of(P, u.r0 + u.rows - 1);
    u.hi = P.causal ? min(s.len, start + i1 + 1) : s.len;
    u.all_hi = P.causal ? min(s.len, start + i0 + 1) : s.len;
    u.lo = seen_from(P, start + i0);
    u.all_lo = seen_from(P, start + i1);
    u.from = w.from;
    u.jb = w.tile;
    u.je = u.hi > u.lo ? w.tile + u.nt : w.tile;
    return u;
}

// A warp's sum of v, and for each lane what is before it.
__device__ __forceinline__ long long scan(long long v, int lane, long long &before) {
    long long x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    before = x - v;
    return __shfl_sync(0xffffffffu, x, 31);
}

// Tiles of the sequences b0 .. b0 + 31, each lane's own.  Blocks of long ones are
// counted by all lanes together.
template <int R>
__device__ __forceinline__ long long seq_tiles(const AttnParams &P, int b0, int lane, bool report) {
    Seq s;
    s.units = 0;
    if (b0 + lane < P.B && !load_seq<R>(P, b0 + lane, s) && report) atomicOr(P.status, STATUS_INDEX);
    long long mine = 0;
    int from;
    const bool far = s.units > 0 && s.blocks > 8;
    if (s.units > 0 && !far)
        for (int k = 0; k < s.blocks; ++k) mine += block_tiles<R>(P, s, k, from);
    for (uint32_t todo = __ballot_sync(0xffffffffu, far); todo; todo &= todo - 1) {
        const int src = __ffs(todo) - 1;
        Seq o;
        o.n = __shfl_sync(0xffffffffu, s.n, src), o.len = __shfl_sync(0xffffffffu, s.len, src);
        const int blocks = __shfl_sync(0xffffffffu, s.blocks, src);
        long long v = 0, before;
        for (int k = lane; k < blocks; k += 32) v += block_tiles<R>(P, o, k, from);
        v = scan(v, lane, before);
        if (lane == src) mine = v;
    }
    return mine * P.heads;
}

// Where this CTA's share begins and ends (see begin_walk for the other kernel).
template <int R>
__device__ __forceinline__ bool begin_rows(const AttnParams &P, int lane, RowWalk &w, long long &t1, long long &W, int &blocks) {
    long long mine = 0, before = 0;
    W = 0;
    for (int b0 = 0; b0 < P.B; b0 += 32) {
        mine = seq_tiles<R>(P, b0, lane, true);
        W += scan(mine, lane, before);
    }
    if (W == 0) return false;
    blocks = static_cast<int>(min(static_cast<long long>(gridDim.x), max(1ll, W / LEAST)));
    const int cta = blockIdx.x;
    if (cta >= blocks) return false;
    t1 = divide((cta + 1) * W, blocks);
    w.t = divide(cta * W, blocks);
    w.u0 = 0;
    for (int b0 = 0;; b0 += 32) {
        if (P.B > 32) mine = seq_tiles<R>(P, b0, lane, false);
        const long long all = scan(mine, lane, before);
        if (w.t < w.u0 + all) {
            const int from = __ffs(__ballot_sync(0xffffffffu, w.t < w.u0 + before + mine)) - 1;
            w.b = b0 + from;
            w.u0 += __shfl_sync(0xffffffffu, before, from);
            break;
        }
        w.u0 += all;
    }
    load_seq<R>(P, w.b, w.s);
    for (int k0 = 0;; k0 += 32) {
        int from;
        mine = k0 + lane < w.s.blocks ? static_cast<long long>(block_tiles<R>(P, w.s, k0 + lane, from)) * P.heads : 0;
        const long long all = scan(mine, lane, before);
        if (w.t < w.u0 + all) {
            const int at = __ffs(__ballot_sync(0xffffffffu, w.t < w.u0 + before + mine)) - 1;
            w.block = k0 + at;
            w.u0 += __shfl_sync(0xffffffffu, before, at);
            break;
        }
        w.u0 += all;
    }
    w.tiles = block_tiles<R>(P, w.s, w.block, w.from);
    w.head = static_cast<int>(divide(w.t - w.u0, w.tiles));
    w.u0 += static_cast<long long>(w.head) * w.tiles;
    w.tile = static_cast<int>(w.t - w.u0);
    if (w.tile && w.tiles <= SHORT) advance<R>(P, w, w.tiles - w.tile, t1);
    return true;
}

// Two values as fp16, and what that leaves of them.
__device__ __forceinline__ uint32_t split2(float a, float b, uint32_t &low) {
    const __half2 h = __floats2half2_rn(a, b);
    const float2 f = __half22float2(h);
    const __half2 l = __floats2half2_rn(a - f.x, b - f.y);
    low = *reinterpret_cast<const uint32_t *>(&l);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// A tile's share of two rows' sums (far_scale), from scores of its own, before the tile's other
// scores take their registers (behind them 1024 rows of 4096 tokens took 335 us instead of 328, as the kernel then was).
template <class C>
__device__ __forceinline__ void far_tile(FarSum *apart, uint32_t sk, const uint4 *my_q, const float *scales, int tok, float4 f, int4 seen) {
#pragma unroll 1
    for (int t = 0; t < TS; ++t) {
        float y[2][4] = {};
#pragma unroll 1
        for (int k = 0; k < C::SIDE / TILE / 16; k += 2) {
            uint32_t a[4];
            ldsm4((sk ^ (k << 4)) + 16 * t * C::ROW, a);
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // two parts of two groups of 16 dims
                const uint4 q = my_q[64 * (k + (i >> 1)) + 32 * (i & 1)];
                const uint32_t qa[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int n = 0; n < 2; ++n) mma16816(y[n], qa, halves(a[(i >> 1) + 2 * n]), halves_hi(a[(i >> 1) + 2 * n]));
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float fk = (h ? f.y : f.x) * scales[t], ek = (h ? f.w : f.z) * scales[t];
            const int lo = h ? seen.y : seen.x, hi = h ? seen.w : seen.z;
            apart[h].add(4, L_FACTOR * 0x1p14f, [&](int i) {
                const int k = tok + 16 * t + 8 * (i >> 1) + (i & 1);
                const float v = y[i >> 1][2 * h + (i & 1)];
                return k >= lo && k < hi ? fmaf(v, fk, v * ek) : -INFINITY;
            });
        }
    }
}

template <int DP>
__global__ void __launch_bounds__(ROWS_THREADS, 1)
    kv_attention_rows_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const AttnParams P) {
    using C = Rows<DP>;
    constexpr int R = C::R, STAGES = C::STAGES, KS = DP / 16;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = smem_u32(smem);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31, g = lane >> 2, c = lane & 3;
    float *const sc = reinterpret_cast<float *>(smem + C::OFF_SC);
    const uint32_t full = base + C::OFF_BAR, empty = full + 8 * STAGES;
    volatile unsigned *const arrived = reinterpret_cast<volatile unsigned *>(smem + C::OFF_BAR + 16 * STAGES);
    volatile unsigned *const some_nan = arrived + 1;  // a NaN among values that not all rows see, in some unit up to here

    if (tid == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, WARPS);
        }
        fence_mbar_init();
        *some_nan = 0;
    }
    pdl_wait();
    pdl_trigger();

    RowWalk w;
    long long t1, W;
    int blocks;
    if (!begin_rows<R>(P, lane, w, t1, W, blocks)) return;
    __syncthreads();  // (the barriers are ready)

    if (warp >= WARPS) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_COPY));
        if (warp == WARPS) copy_tiles<C>(P, tmK, tmV, w, t1, blockIdx.x == 0 ? P.stop : NO_STOP, base, sc, full, empty, lane);
        return;
    }
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_ROWS));

    // this lane's fragments of the queries, which nobody else reads
    uint4 *const my_q = reinterpret_cast<uint4 *>(smem + C::OFF_Q + warp * C::Q_WARP) + lane;
    const bool vec = ((reinterpret_cast<uintptr_t>(P.q) & 15) | ((P.ldq_t | P.ldq_h) & 3)) == 0;
    int it = 0;
    bool dead = false;  // a wait ran out: this warp only goes through the barriers from here on
    while (w.t < t1) {
        const Span u = span_of<R>(P, w, t1);
        const Seq &s = w.s;
        const int r0 = u.r0, rows = u.rows, head = u.head, start = s.len - s.n;
        const bool idle = 16 * warp >= rows;

        // this lane's rows g and g + 8 of the warp's (those behind the last one: copies of it)
        float f[2], f_low[2];
        int lo[2], hi[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int qr = r0 + min(16 * warp + g + 8 * h, rows - 1), i = token_of(P, qr);
            hi[h] = P.causal ? min(s.len, start + i + 1) : s.len;
            lo[h] = seen_from(P, start + i);
            const float *const q = static_cast<const float *>(P.q) + (static_cast<int64_t>(s.row0) + i) * P.ldq_t +
                                   static_cast<int64_t>(head * P.group + (qr - i * P.group)) * P.ldq_h;
            float4 v[KS];
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const int d = 16 * k + 4 * c;
                v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (16 * k < P.dim) {
                    if (vec) v[k] = __ldg(reinterpret_cast<const float4 *>(q + d));
                    else v[k] = make_float4(__ldg(q + d), __ldg(q + d + 1), __ldg(q + d + 2), __ldg(q + d + 3));
                }
            }
            // times a power of two that brings the largest to [2^13, 2^14)
            float top = 0.0f;
            auto most = [&](float a) { top = fabsf(a) <= 3.402823466e38f ? fmaxf(top, fabsf(a)) : top; };
#pragma unroll
            for (int k = 0; k < KS; ++k) most(v[k].x), most(v[k].y), most(v[k].z), most(v[k].w);
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int e = top > 0.0f ? min(max(13 - exponent_of(__float_as_uint(top)), -114), 100) : 0;
            const float up = pow2f(e);
            f[h] = P.factor * pow2f(-e), f_low[h] = P.factor_low * pow2f(-e);
            auto scaled = [&](float a) { return a * up + (a - a); };  // (an infinity as NaN)
            uint32_t *const sq = reinterpret_cast<uint32_t *>(my_q);
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                uint32_t low;
                sq[256 * k + h] = split2(scaled(v[k].x), scaled(v[k].y), low), sq[256 * k + 128 + h] = low;
                sq[256 * k + 2 + h] = split2(scaled(v[k].z), scaled(v[k].w), low), sq[256 * k + 130 + h] = low;
            }
        }
        // tokens that some of the warp's rows see
        const int some_hi = __reduce_max_sync(0xffffffffu, max(hi[0], hi[1]));
        const int some_lo = __reduce_min_sync(0xffffffffu, min(lo[0], lo[1]));

        float o[DP / 8][4];
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
        for (int n = 0; n < DP / 8; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[n][i] = 0.0f;

        FarSum apart[2];
        bool far = false;
        for (int j = u.jb; j < u.je; ++j, ++it) {
            const int slot = it % STAGES;
            if (!dead) dead = !__all_sync(0xffffffffu, mbar_wait(full + 8 * slot, (it / STAGES) & 1, P.status));
            // (a row's 16-byte chunks lie in the order of its swizzle: another chunk is an exclusive or away)
            const uint32_t sk = base + slot * C::STAGE + C::at((lane & 7) + (lane >> 4 << 3), lane >> 3 & 1);
            const uint32_t sv = base + slot * C::STAGE + C::SIDE + C::at(lane & 15, lane >> 4);
            const int tok0 = u.from + j * TILE;
            if (!dead && !idle && sc[SCALES * slot + 16] == 0.0f) {  // the sums apart (far_scale)
                if (!far) apart[0].m = m[0], apart[0].l = l[0], apart[1].m = m[1], apart[1].l = l[1];
                far = true;
                far_tile<C>(apart, sk, my_q, sc + SCALES * slot, tok0 + 2 * c, make_float4(f[0], f[1], f_low[0], f_low[1]),
                            make_int4(lo[0], lo[1], hi[0], hi[1]));
            }
            const bool whole = tok0 >= u.all_lo && tok0 + TILE <= u.all_hi;  // (the same for all warps)
            if (!whole) {
                // What no row sees counts as 0, and so does a NaN for now: as in
                // kv_attention.cuh, each warp for 16 tokens.
                if (!dead) {
                    uint8_t *const values = smem + slot * C::STAGE + C::SIDE;
#pragma unroll 1
                    for (int i = 0; i < 16 * KS / 32; ++i) {
                        const int row = 16 * warp + (32 * i + lane) / KS;
                        uint4 *v = reinterpret_cast<uint4 *>(values + C::at(row, (32 * i + lane) % KS));
                        const bool seen = tok0 + row >= u.lo && tok0 + row < u.hi, bad = seen && has_nan(*v);
                        if (!seen) *v = make_uint4(0, 0, 0, 0);
                        if (bad) *v = without_nan(*v), *some_nan = 1;
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // (before the next copy into the slot)
                }
                named_barrier(1, C::CONSUMERS);
            }
            if (!dead && !idle && tok0 < some_hi && tok0 + TILE > some_lo) {
                // S
                float x[2 * TS][4];
#pragma unroll
                for (int n = 0; n < 2 * TS; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[n][i] = 0.0f;
#pragma unroll
                for (int k = 0; k < KS; k += 2) {
                    uint32_t qh[2][4], ql[2][4];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint4 a = my_q[64 * (k + h)], b = my_q[64 * (k + h) + 32];
                        qh[h][0] = a.x, qh[h][1] = a.y, qh[h][2] = a.z, qh[h][3] = a.w;
                        ql[h][0] = b.x, ql[h][1] = b.y, ql[h][2] = b.z, ql[h][3] = b.w;
                    }
#pragma unroll
                    for (int t = 0; t < TS; t += 2) {
                        uint32_t a[2][4];  // of 16 tokens: 8 and 8, of two groups of 16 dims
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            ldsm4((sk ^ (k << 4)) + 16 * (t + i) * C::ROW, a[i]);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t b[4][2];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const uint32_t codes = a[i >> 1][h + 2 * (i & 1)];
                                b[i][0] = halves(codes), b[i][1] = halves_hi(codes);
                            }
#pragma unroll
                            for (int i = 0; i < 4; ++i) mma16816(x[2 * t + i], qh[h], b[i][0], b[i][1]);
#pragma unroll
                            for (int i = 0; i < 4; ++i) mma16816(x[2 * t + i], ql[h], b[i][0], b[i][1]);
                        }
                    }
                }
                // P, the operand of the second product.  Masks only where the
                // unit's rows do not all see the tile: an instance of its own.
                uint32_t ph[TS][4], pl[TS][4];
                float alpha[2];
                auto softmax = [&](auto masked) {
                    constexpr bool MASKED = decltype(masked)::value;
                    uint32_t hidden[TS] = {};  // bit 4 b + i of t: x[2 t + b][i] is masked
                    if constexpr (MASKED) {
#pragma unroll
                        for (int n = 0; n < 2 * TS; ++n)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int tok = tok0 + 8 * n + 2 * c + (i & 1);
                                if (tok < lo[i >> 1] || tok >= hi[i >> 1]) hidden[n >> 1] |= 1u << (4 * (n & 1) + i);
                            }
                    }
                    const float *const scales = sc + SCALES * slot;
                    float top[2] = {m[0], m[1]};
#pragma unroll
                    for (int t = 0; t < TS; ++t) {
                        const float ks = scales[t], lv = scales[8 + t], fk[2] = {f[0] * ks, f[1] * ks};
#pragma unroll
                        for (int b = 0; b < 2; ++b)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                float y = fmaf(x[2 * t + b][i], fk[i >> 1], lv);
                                if (MASKED && hidden[t] >> (4 * b + i) & 1) y = -INFINITY;
                                top[i >> 1] = fmaxf(top[i >> 1], y);
                            }
                    }
                    float ref[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
                        top[h] = ceilf(fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2)));  // (a whole number: see there)
                        ref[h] = top[h] == -INFINITY ? 0.0f : top[h];  // (a row that has seen nothing yet: any finite one)
                        alpha[h] = ex2(m[h] - ref[h]);
                        m[h] = top[h];
                        l[h] *= alpha[h];
                    }
#pragma unroll
                    for (int t = 0; t < TS; ++t) {
                        const float ks = scales[t], lv = scales[8 + t], iv = scales[16 + t] * L_FACTOR;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float fk = f[h] * ks, ek = f_low[h] * ks, shift = (lv - ref[h]) + P_SHIFT;
                            float sum = 0.0f;
#pragma unroll
                            for (int b = 0; b < 2; ++b) {
                                float p[2];
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    const float v = x[2 * t + b][2 * h + i];
                                    p[i] = ex2(fmaf(v, fk, fmaf(v, ek, shift)));
                                    if (MASKED && hidden[t] >> (4 * b + 2 * h + i) & 1) p[i] = 0.0f;
                                }
                                sum += p[0] + p[1];
                                ph[t][2 * b + h] = split2(p[0], p[1], pl[t][2 * b + h]);
                            }
                            l[h] = fmaf(sum, iv, l[h]);
                        }
                    }
                };
                if (whole) softmax(std::false_type{});
                else softmax(std::true_type{});
                // O: dims 32 d + 16 n + 4 c .. + 3 of the rows, even ones and odd ones
#pragma unroll
                for (int d = 0; d < DP / 32; ++d) {
                    float acc[4][4];
#pragma unroll
                    for (int n = 0; n < 4; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;
#pragma unroll
                    for (int t = 0; t < TS; ++t) {
                        uint32_t a[4];
                        ldsm4_t((sv ^ (d << 5)) + 16 * t * C::ROW, a);
                        uint32_t b[4][2];
#pragma unroll
                        for (int n = 0; n < 2; ++n)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const uint32_t codes = __byte_perm(a[2 * n + i], 0, 0x3120);
                                b[2 * n][i] = halves(codes), b[2 * n + 1][i] = halves_hi(codes);
                            }
#pragma unroll
                        for (int n = 0; n < 4; ++n) mma16816(acc[n], ph[t], b[n][0], b[n][1]);
#pragma unroll
                        for (int n = 0; n < 4; ++n) mma16816(acc[n], pl[t], b[n][0], b[n][1]);
                    }
#pragma unroll
                    for (int n = 0; n < 4; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[4 * d + n][i] = fmaf(o[4 * d + n][i], alpha[i >> 1], acc[n][i]);
                }
            }
            __syncwarp();
            if (lane == 0 && !dead) mbar_arrive(empty + 8 * slot);
        }
        // (where a warp has skipped every tile its l is 0 in either way)
        if (far) l[0] = apart[0].at(m[0]), l[1] = apart[1].at(m[1]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        }

        auto out = [&](int r, int64_t &at, int64_t &row) {
            const int i = token_of(P, r0 + r), h = head * P.group + (r0 + r - i * P.group);
            at = (static_cast<int64_t>(s.row0) + i) * P.ldy_t + static_cast<int64_t>(h) * P.ldy_h;
            row = (static_cast<int64_t>(s.row0) + i) * P.heads * P.group + h;
        };
        const bool entire = u.nt == w.tiles;
        // (an entire unit's results, or a part of it: [row][dim] sums relative to m, then m and l)
        float *const mine = P.part + (static_cast<int64_t>(blockIdx.x) * 2 + (w.tile == 0)) * C::PART;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = 16 * warp + g + 8 * h;
            if (r >= rows) continue;
            int64_t at = 0, row = 0;
            if (entire) out(r, at, row);
            const float inv = l[h] != 0.0f ? L_FACTOR / l[h] : 0.0f;
#pragma unroll
            for (int n = 0; n < DP / 16; ++n) {
                const int d = 16 * n + 4 * c;
                const float4 v = make_float4(o[2 * n][2 * h], o[2 * n + 1][2 * h], o[2 * n][2 * h + 1], o[2 * n + 1][2 * h + 1]);
                if (!entire) {
                    *reinterpret_cast<float4 *>(mine + r * DP + d) = v;
                } else if (d < P.dim) {
                    store_typed(P.y, at + d, P.y_type, v.x * inv);
                    store_typed(P.y, at + d + 1, P.y_type, v.y * inv);
                    store_typed(P.y, at + d + 2, P.y_type, v.z * inv);
                    store_typed(P.y, at + d + 3, P.y_type, v.w * inv);
                }
            }
            if (!entire && c == 0) mine[R * DP + r] = m[h], mine[R * (DP + 1) + r] = l[h];
            if (entire && P.lse && c == 0) P.lse[row] = l[h] != 0.0f ? (m[h] + log2f(l[h]) + 20.0f - C::SHIFT) * LN2 : -INFINITY;
        }
        // (every tile that not all rows see had a barrier behind the search)
        if (__any_sync(0xffffffffu, *some_nan != 0)) {
            __syncwarp();  // (other lanes wrote what these change; a vote orders no memory)
            spread_nans(P, w.b, head, start, r0, 16 * warp, min(rows, 16 * warp + 16), 0, DP, max(u.from + u.jb * TILE, u.lo),
                        min(u.from + u.je * TILE, u.hi), u.all_lo, u.all_hi, lane, 32, [&](int r, int d) {
                            int64_t at, row;
                            out(r, at, row);
                            if (entire) store_typed(P.y, at + d, P.y_type, __uint_as_float(A_NAN));
                            else mine[r * DP + d] = __uint_as_float(A_NAN);
                        });
        }
        if (!entire) {
            far = named_barrier_or(1, C::CONSUMERS, far);
            // the CTAs of the unit's first and last tile
            const int c0 = static_cast<int>(divide((w.u0 + 1) * blocks - 1, W)), c1 = static_cast<int>(divide((w.u0 + w.tiles) * blocks - 1, W));
            if (tid == 0) *arrived = arrive(P.count + c0, static_cast<unsigned>(c1 - c0), far);
            named_barrier(1, C::CONSUMERS);
            const unsigned parts = *arrived;
            if ((parts & (FAR_PART - 1)) == static_cast<unsigned>(c1 - c0)) join_parts<C, DP>(P, c0, c1, rows, tid, parts >= FAR_PART, out);
        }
        advance<R>(P, w, u.nt, t1);
    }
}

template <int DP>
cudaError_t launch_dp(const AttnParams &p, cudaStream_t st, int num_sms, int dev) {
    using C = Rows<DP>;
    const auto kern = kv_attention_rows_kernel<DP>;
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
    cfg.blockDim = dim3(ROWS_THREADS);
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

size_t rows_part_bytes(int dim, int num_sms) {
    return static_cast<size_t>(num_sms) * 2 * 4 * (dim <= 64 ? Rows<64>::PART : Rows<128>::PART);
}

cudaError_t launch_rows(const AttnParams &p, cudaStream_t st, int num_sms, int dev) {
    return p.dim <= 64 ? launch_dp<64>(p, st, num_sms, dev) : launch_dp<128>(p, st, num_sms, dev);
}

}  // namespace kv
}  // namespace qk
