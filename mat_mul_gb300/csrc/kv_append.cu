// kv_append.cu -- new rows of keys and values into the paged cache as e4m3
// codes, the keys (and the queries beside them) turned by their positions on
// the way.
//
// A page of one head has one scale s, a power of two: the smallest at which
// the largest |value| is at most 448 s.  It only grows while tokens are added
// to a page, and the codes that the page holds are then rounded anew (by a power
// of two, so only what falls below the normal codes loses anything); the first
// token of a page starts it afresh.  A block owns the rows of one page of one
// head: it takes their maximum, so nobody else writes the page's scale, and
// nothing depends on the order of blocks.  For prompts a block takes several heads
// one after another, the next one's rows on their way meanwhile: finding the page
// takes four dependent loads, and the sines are the same for all heads (8247 rows
// of 8 heads of 128: 30 us with a block per head).
//
// Bound by memory for a prompt (every row read once, its codes written once),
// by latency for single tokens.  8247 rows of 40 + 2 x 8 heads of 128 bf16, queries turned
// beside: 42 us, 0.77 of the rate of a copy.
#include "kv_device.cuh"

namespace qk {

namespace {

struct AppendParams {
    uint8_t *codes[2];  // of keys, of values
    float *scales[2];
    int64_t pages;
    int heads, page, dim, q_heads, q_per, kv_per;  // .._per: heads of a block
    const void *x[3];  // new keys, values and queries
    int64_t ld_t[3], ld_h[3];
    void *y;
    int64_t ldy_t, ldy_h;
    const int32_t *offsets, *lengths, *table, *positions;
    int64_t ld_table, T;
    int width, B;
    RopeArgs rope;
    int *status;
};

// Rows `row` .. `row + n) of the batch, tokens `pos` .. of their sequence, all in one page.
struct Unit {
    int64_t row;
    int pos, n, page;
};

// The unit u of the launch: sequence b has the units from offsets[b] / page + 2 b
// on, which are enough for its rows (they lie in at most (n - 1) / page + 2
// pages) and need no sum over the sequences before it.  False where there is none.
// The lanes of a warp search together, 32 sequences at a time.
__device__ bool find_unit(const AppendParams &P, int u, Unit &q) {
    int b = u, lo = u, n = 1, ordinal = 0;
    if (P.offsets) {
        const int lane = threadIdx.x & 31;
        int first = 0, count = P.B, begin = 0;  // the last sequence that begins at u or before it is one of `count` from `first` on
        for (;;) {
            const int step = (count + 31) / 32, i = first + lane * step;
            int off = 0;
            if (lane * step < count) off = __ldg(P.offsets + i);
            const unsigned at = __ballot_sync(0xffffffffu, lane * step < count && off / P.page + 2 * i <= u);
            const int last = at ? 31 - __clz(at) : 0;
            first += last * step;
            begin = __shfl_sync(0xffffffffu, off, last);
            if (step == 1) break;
            count = min(step, count - last * step);
        }
        b = first;
        lo = begin;
        const int hi = __ldg(P.offsets + b + 1);
        if (lo < 0 || hi < lo || hi > P.T) {
            atomicOr(P.status, STATUS_INDEX);
            return false;
        }
        n = hi - lo;
        ordinal = u - (lo / P.page + 2 * b);
        if (n == 0 || ordinal < 0) return false;
    }
    const int len = __ldg(P.lengths + b);
    if (len < n || len > static_cast<int64_t>(P.width) * P.page) {
        atomicOr(P.status, STATUS_INDEX);
        return false;
    }
    const int start = len - n;
    const int64_t ord = start / P.page + ordinal;
    const int64_t p0 = max(static_cast<int64_t>(start), ord * P.page), p1 = min(static_cast<int64_t>(len), (ord + 1) * P.page);
    if (p0 >= p1) return false;
    q.page = __ldg(P.table + b * P.ld_table + ord);
    q.row = lo + (p0 - start);
    q.pos = static_cast<int>(p0);
    q.n = static_cast<int>(p1 - p0);
    return true;
}

constexpr float LARGEST = 3.402823466e38f;

// Codes of values times inv; a NaN has one.
__device__ __forceinline__ uint32_t codes2(float a, float b, float inv) {
    return __nv_cvt_float2_to_fp8x2(make_float2(a * inv, b * inv), __NV_SATFINITE, __NV_E4M3);
}
template <int V>
__device__ __forceinline__ void store_codes(uint8_t *p, const float *v, float inv) {
    if constexpr (V == 1) {
        *p = static_cast<uint8_t>(codes2(v[0], 0.0f, inv));
    } else {
        *reinterpret_cast<uint32_t *>(p) = codes2(v[0], v[1], inv) | codes2(v[2], v[3], inv) << 16;
    }
}

// Four codes times `ratio`, rounded anew.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio) {
    uint32_t out = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> (16 * i)), __NV_E4M3);
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        out |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(f.x * ratio, f.y * ratio), __NV_SATFINITE,
                                                              __NV_E4M3))
               << (16 * i);
    }
    return out;
}

// KEEP groups of a thread stay in registers between the maximum and the codes;
// with KEEP = 0 they are read and turned twice.
// QV: pairs of a group of the queries.
template <int T, int V, int QV, int THREADS, int KEEP>
__global__ void __launch_bounds__(THREADS, THREADS == 256 && KEEP <= 4 ? 2 : 1) kv_append_kernel(const AppendParams P) {
    using X = typename KvElem<T>::type;
    __shared__ float reduced[2][THREADS / 32 + 1];
    pdl_wait();
    pdl_trigger();
    // Offsets that fall can hide a sequence from every search, and another's units behind
    // it: block u looks at those of sequence u as well (there are more units than
    // sequences).  Loaded before the search, so that nothing waits for them.
    const bool check = P.offsets && blockIdx.y == 0 && blockIdx.x < static_cast<unsigned>(P.B);
    int lo = 0, hi = 0;
    if (check) lo = __ldg(P.offsets + blockIdx.x), hi = __ldg(P.offsets + blockIdx.x + 1);
    Unit u;
    const bool have = find_unit(P, blockIdx.x, u);
    if (check && threadIdx.x == 0 && (lo < 0 || hi < lo || hi > P.T)) atomicOr(P.status, STATUS_INDEX);
    if (!have) return;
    const int tid = threadIdx.x, kv_parts = (P.heads + P.kv_per - 1) / P.kv_per, part = blockIdx.y;
    if (part >= 2 * kv_parts) {  // queries
        const int h0 = (part - 2 * kv_parts) * P.q_per, h1 = min(P.q_heads, h0 + P.q_per);
        const int q_groups = P.dim / (2 * QV);
        for (int i = tid; i < u.n * q_groups; i += THREADS) {
            const int t = i / q_groups;
            const Group<QV> group(i - t * q_groups, P.rope);
            const int64_t row = u.row + t;
            float2 cs[QV];
            group.angles(P.rope, P.positions ? __ldg(P.positions + row) : u.pos + t, cs);
            turn_heads<X, X, QV, 4>(static_cast<const X *>(P.x[2]) + row * P.ld_t[2] + h0 * P.ld_h[2], P.ld_h[2],
                                    static_cast<X *>(P.y) + row * P.ldy_t + h0 * P.ldy_h, P.ldy_h, h1 - h0, group, cs);
        }
        return;
    }
    if (u.page < 0 || u.page >= P.pages) {
        atomicOr(P.status, STATUS_INDEX);
        return;
    }
    const int is_v = part >= kv_parts, h0 = (part - is_v * kv_parts) * P.kv_per, h1 = min(P.heads, h0 + P.kv_per);
    RopeArgs rope = P.rope;
    if (is_v) rope.rot = 0;
    const int slot = u.pos % P.page;
    const int64_t tile0 = static_cast<int64_t>(u.page) * P.heads;
    int turn = 0;

    // A thread has one group of every `step`th row.
    const int groups = P.dim / (2 * V), step = THREADS / groups, row0 = tid / groups;
    const int n = row0 < step && tid < THREADS ? u.n : 0;
    const Group<V> group(tid - row0 * groups, rope);
    auto source = [&](int h, int t, Run<X, V> (&r)[2]) {
        const X *p = static_cast<const X *>(P.x[is_v]) + (u.row + t) * P.ld_t[is_v] + h * P.ld_h[is_v];
        r[0] = load_run<X, V>(p + group.first), r[1] = load_run<X, V>(p + group.second);
    };
    auto angles = [&](int t, float2 (&cs)[V]) { group.angles(rope, P.positions ? __ldg(P.positions + u.row + t) : u.pos + t, cs); };
    auto values = [&](const Run<X, V> (&r)[2], const float2 (&cs)[V], float (&v)[2 * V]) {
        values_of<X, V>(r[0], v), values_of<X, V>(r[1], v + V);
        group.turn(v, cs);
    };
    auto largest = [](float a, const float (&v)[2 * V]) {
#pragma unroll
        for (int j = 0; j < 2 * V; ++j) a = fmaxf(a, fabsf(v[j]));  // (passes over NaNs)
        return a;
    };
    // (an infinity has no code: it becomes a NaN)
    auto finite = [](float (&v)[2 * V]) {
#pragma unroll
        for (int j = 0; j < 2 * V; ++j) v[j] = fabsf(v[j]) <= LARGEST ? v[j] : __uint_as_float(0x7fffffffu);
    };
    auto block_max = [&](float top) {
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if constexpr (THREADS > 32) {
            float *const red = reduced[turn];  // (the next barrier lies before this half is used again)
            turn ^= 1;
            if ((tid & 31) == 0) red[tid >> 5] = top;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < THREADS / 32; ++w) top = fmaxf(top, red[w]);
        } else {
            __syncwarp();
        }
        return top;
    };
    // The page's new scale of head h, after what the page holds was rounded to it:
    // the smallest power of two s with top <= 448 s, or the old one.  Every thread
    // has read the old one (`before`) ahead of the barrier of the maximum.
    auto rescale = [&](int h, float top, float before) {
        // top <= 1.75 * 2^8 of it: one power more where the mantissa of top is above 1.75
        const int e = max(static_cast<int>((__float_as_uint(top) + 0x1fffffu) >> 23) - 127 - 8, KV_LEAST_EXP);
        const float s = fmaxf(pow2f(e), before);
        if (s != before) {
            if (tid == 0) P.scales[is_v][tile0 + h] = s;
            if (slot) {
                const float ratio = before * __fdiv_rn(1.0f, s);
                uint4 *w = reinterpret_cast<uint4 *>(P.codes[is_v] + (tile0 + h) * P.page * P.dim);
                for (int i = tid; i < slot * P.dim / 16; i += THREADS) {
                    const uint4 q = w[i];
                    w[i] = make_uint4(rescale4(q.x, ratio), rescale4(q.y, ratio), rescale4(q.z, ratio), rescale4(q.w, ratio));
                }
            }
        }
        return __fdiv_rn(1.0f, s);
    };
    auto put = [&](int h, int t, const float (&w)[2 * V], float inv) {
        uint8_t *codes = P.codes[is_v] + ((tile0 + h) * P.page + slot + t) * P.dim;
        store_codes<V>(codes + group.first, w, inv);
        store_codes<V>(codes + group.second, w + V, inv);
    };
    auto scale_of = [&](int h) { return slot ? P.scales[is_v][tile0 + h] : 0.0f; };

    if constexpr (KEEP > 0) {
        // the sines of a thread's rows, for all heads (with more than four they are found again for each)
        constexpr bool SAME = KEEP <= 4;
        float2 cs[SAME ? KEEP : 1][V];
        Run<X, V> r[KEEP][2];
#pragma unroll
        for (int k = 0; k < KEEP; ++k) source(h0, min(row0 + k * step, u.n - 1), r[k]);  // (all of them on their way at once)
        float before = scale_of(h0);
        if constexpr (SAME) {
#pragma unroll
            for (int k = 0; k < KEEP; ++k) angles(min(row0 + k * step, u.n - 1), cs[k]);
        }
        for (int h = h0; h < h1; ++h) {
            float v[KEEP][2 * V];
            float top = 0.0f;
#pragma unroll
            for (int k = 0; k < KEEP; ++k)
                if (row0 + k * step < n) {
                    if constexpr (!SAME) angles(row0 + k * step, cs[0]);
                    values(r[k], cs[SAME ? k : 0], v[k]);
                    top = largest(top, v[k]);
                }
            const float old = before;
            if (h + 1 < h1) {
#pragma unroll
                for (int k = 0; k < KEEP; ++k) source(h + 1, min(row0 + k * step, u.n - 1), r[k]);
                before = scale_of(h + 1);
            }
            top = block_max(top);
            if (top > LARGEST) {
                top = 0.0f;
#pragma unroll
                for (int k = 0; k < KEEP; ++k)
                    if (row0 + k * step < n) {
                        finite(v[k]);
                        top = largest(top, v[k]);
                    }
                top = block_max(top);
            }
            const float inv = rescale(h, top, old);
#pragma unroll
            for (int k = 0; k < KEEP; ++k)
                if (row0 + k * step < n) put(h, row0 + k * step, v[k], inv);
        }
    } else {
        for (int h = h0; h < h1; ++h) {
            const float before = scale_of(h);
            float inv = 0.0f;
            for (int pass = 0; pass < 2; ++pass) {
                float top = 0.0f;
                // (this path has several groups per thread: `groups` may exceed THREADS)
                for (int i = tid; i < u.n * groups; i += THREADS) {
                    const int t = i / groups;
                    const Group<V> g(i - t * groups, rope);
                    const X *p = static_cast<const X *>(P.x[is_v]) + (u.row + t) * P.ld_t[is_v] + h * P.ld_h[is_v];
                    float2 cs[V];
                    float v[2 * V];
                    g.angles(rope, P.positions ? __ldg(P.positions + u.row + t) : u.pos + t, cs);
                    values_of<X, V>(load_run<X, V>(p + g.first), v), values_of<X, V>(load_run<X, V>(p + g.second), v + V);
                    g.turn(v, cs);
                    finite(v);
                    if (pass) {
                        uint8_t *codes = P.codes[is_v] + ((tile0 + h) * P.page + slot + t) * P.dim;
                        store_codes<V>(codes + g.first, v, inv);
                        store_codes<V>(codes + g.second, v + V, inv);
                    } else {
                        top = largest(top, v);
                    }
                }
                if (!pass) inv = rescale(h, block_max(top), before);
            }
        }
    }
}

template <int T, int V, int QV, int THREADS, int KEEP>
cudaError_t launch_one(const AppendParams &p, unsigned units, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(units, static_cast<unsigned>(2 * ((p.heads + p.kv_per - 1) / p.kv_per) + (p.q_heads ? (p.q_heads + p.q_per - 1) / p.q_per : 0)));
    cfg.blockDim = dim3(THREADS);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv_append_kernel<T, V, QV, THREADS, KEEP>, p);
}

template <int T, int QV>
cudaError_t launch_keep(const AppendParams &p, unsigned units, cudaStream_t st) {
    if (!p.offsets) return launch_one<T, 4, QV, 32, 1>(p, units, st);
    // rows of a thread: KEEP hold a page's
    auto rows = [&](int threads) { return (p.page + threads / (p.dim / 8) - 1) / (threads / (p.dim / 8)); };
    if (rows(256) <= 4) return launch_one<T, 4, QV, 256, 4>(p, units, st);
    if (rows(256) <= 8) return launch_one<T, 4, QV, 256, 8>(p, units, st);
    return launch_one<T, 4, QV, 512, 8>(p, units, st);  // (8 for heads of 256 values and pages of 128 tokens, fewer below)
}

// runs: values that the rows allow to take at once.
template <int T>
cudaError_t launch_t(const AppendParams &p, int runs, unsigned units, cudaStream_t st) {
    if (runs < 4) return p.offsets ? launch_one<T, 1, 1, 256, 0>(p, units, st) : launch_one<T, 1, 1, 32, 0>(p, units, st);
    if constexpr (T != QMM_F32)
        if (runs == 8 && p.q_heads) return launch_keep<T, 8>(p, units, st);
    return launch_keep<T, 4>(p, units, st);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppend &a, cudaStream_t st, int num_sms) {
    AppendParams p = {};
    p.codes[0] = static_cast<uint8_t *>(a.c.k), p.codes[1] = static_cast<uint8_t *>(a.c.v);
    p.scales[0] = a.c.k_scale, p.scales[1] = a.c.v_scale;
    p.pages = a.c.pages;
    p.heads = static_cast<int>(a.c.heads), p.page = static_cast<int>(a.c.page), p.dim = static_cast<int>(a.c.dim);
    const Heads *in[3] = {&a.k, &a.v, &a.q};
    const int64_t T = a.batch.T;
    auto runs_of = [&](const Heads &h, int heads, int n) {
        const int es = f8_size(h.type);
        return reinterpret_cast<uintptr_t>(h.x) % (n * es) == 0 && (T == 1 || h.ld_t % n == 0) && (heads == 1 || h.ld_h % n == 0);
    };
    p.q_heads = a.q.x ? a.q_heads : 0;
    for (int i = 0; i < 3; ++i) p.x[i] = in[i]->x, p.ld_t[i] = in[i]->ld_t, p.ld_h[i] = in[i]->ld_h;
    auto fits = [&](int n) {
        return a.rope.rot % (2 * n) == 0 && runs_of(a.k, p.heads, 4) && runs_of(a.v, p.heads, 4) &&
               (!a.q.x || (runs_of(a.q, a.q_heads, n) && runs_of(a.y, a.q_heads, n)));
    };
    const int runs = fits(8) ? 8 : fits(4) ? 4 : 1;
    p.y = const_cast<void *>(a.y.x), p.ldy_t = a.y.ld_t, p.ldy_h = a.y.ld_h;
    p.offsets = a.batch.offsets, p.lengths = a.batch.lengths, p.table = a.batch.table, p.positions = a.positions;
    p.ld_table = a.batch.ld_table, p.T = T, p.width = a.batch.width, p.B = a.batch.B;
    p.rope = a.rope;
    p.status = a.status;
    p.q_per = a.batch.offsets ? 8 : 2;
    p.kv_per = a.batch.offsets ? 8 : 1;
    const int64_t units = a.batch.offsets ? T / p.page + 2 * int64_t(p.B) : p.B;
    if (units > 0x7fffffff) return cudaErrorInvalidConfiguration;
    const unsigned n = static_cast<unsigned>(units);
    if (a.k.type == QMM_F32) return launch_t<QMM_F32>(p, runs, n, st);
    if (a.k.type == QMM_F16) return launch_t<QMM_F16>(p, runs, n, st);
    return launch_t<QMM_BF16>(p, runs, n, st);
}

}  // namespace qk
